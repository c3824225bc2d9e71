"""A gated delta rule block served with the framework's layers: a prompt at once, then token by token from
the states it left.

    p         = in_proj(u)                                   pointwise  C -> 2 Hk K + H V | H V | H | H
    q, k, v   = silu(causal depthwise conv(p[:, :2 Hk K + H V]))
    y         = gated delta rule(q, k, v, dt, a, b)          dt, b: p's last columns
    out       = u + out_proj(rms norm of y's heads * silu(z)) pointwise  H V -> C

The pointwise layers are microscaled 4-bit on both sides: weights are quantised once, rows in each call, by
the framework's own kernel.  All layers take prompts and single tokens alike, and hand their states on in
place.  Run: python examples/delta_block.py"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import pointwise_conv_cnn_gb300 as fcm  # noqa: E402

DTYPE = torch.bfloat16


class Pointwise:
    """y = x W^T on rows of tokens, both in microscaled 4-bit values."""

    def __init__(self, w: torch.Tensor):
        self.out, self.inp = w.shape
        self.q, self.s = self.quantised(w)

    @staticmethod
    def quantised(x: torch.Tensor):
        q = torch.empty((x.shape[0], x.shape[1] // 2), dtype=torch.uint8, device=x.device)
        s = torch.empty((x.shape[0], x.shape[1] // 32), dtype=torch.uint8, device=x.device)
        fcm.mx4_quantize(x, q, s)
        return q, s

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        q, s = self.quantised(x)
        y = torch.empty((x.shape[0], self.out), dtype=DTYPE, device=x.device)
        fcm.mx4_matmul(q, s, self.q, self.s, y)
        return y


class DeltaBlock:
    """One block with its states; `slots` sequences can be in flight."""

    def __init__(self, c=128, key_heads=1, heads=2, dk=64, dv=64, taps=4, slots=4, seed=0, device="cuda"):
        g = torch.Generator("cpu").manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(device)
        self.key_heads, self.heads, self.dk, self.dv = key_heads, heads, dk, dv
        self.mixed = 2 * key_heads * dk + heads * dv   # q, k and v side by side
        self.in_proj = Pointwise(normal(self.mixed + heads * dv + 2 * heads, c))
        self.out_proj = Pointwise(normal(c, heads * dv))
        self.conv_w = normal(self.mixed, taps).to(DTYPE)
        self.a = -torch.linspace(1.0, 8.0, heads, device=device)
        self.dt_bias = torch.linspace(-4.0, -2.0, heads, device=device)
        self.norm = torch.linspace(0.5, 1.5, heads * dv, device=device)
        self.conv_state = torch.zeros((slots, taps - 1, self.mixed), dtype=DTYPE, device=device)
        self.state = torch.zeros((slots, heads, dk, dv), device=device)

    def mix(self, p: torch.Tensor, slot: torch.Tensor) -> torch.Tensor:
        """p [sequences, length, columns of in_proj] -> the normalised heads [tokens, H V]."""
        s, length, _ = p.shape
        m, h, keys = self.mixed, self.heads, self.key_heads * self.dk
        x = torch.empty((s, length, m), dtype=DTYPE, device=p.device)
        fcm.causal_conv(p[..., :m], self.conv_w, x, act="silu", slot=slot, state_in=self.conv_state,
                        state_out=self.conv_state)
        q, k = (x[..., i * keys:(i + 1) * keys].unflatten(-1, (self.key_heads, self.dk)) for i in range(2))
        v = x[..., 2 * keys:].unflatten(-1, (h, self.dv))
        at = m + h * self.dv
        y = torch.empty((s, length, h, self.dv), dtype=DTYPE, device=p.device)
        fcm.gated_delta(q, k, v, p[..., at:at + h], self.a, p[..., at + h:], y, dt_bias=self.dt_bias, slot=slot,
                        state_in=self.state, state_out=self.state)
        out = torch.empty((s * length, h * self.dv), dtype=DTYPE, device=p.device)
        fcm.group_norm(y.view(out.shape), out, h, scale=self.norm, z=p.view(s * length, -1)[:, m:at], rms=True)
        return out

    def __call__(self, u: torch.Tensor, slot: torch.Tensor) -> torch.Tensor:
        """u [sequences, length, c]: the next rows of the sequences whose states are in rows `slot`
        (int32 [sequences]); the states move on."""
        s, length, c = u.shape
        p = self.in_proj(u.reshape(-1, c)).view(s, length, -1)
        return u + self.out_proj(self.mix(p, slot)).view(s, length, c)

    def reset(self) -> None:
        self.conv_state.zero_()
        self.state.zero_()


def serve(prompt=50, tokens=12, sequences=2, c=128) -> tuple[torch.Tensor, torch.Tensor]:
    """The same rows once as one prompt, once as a shorter prompt and single tokens."""
    block = DeltaBlock(c=c)
    u = torch.randn((sequences, prompt + tokens, c), generator=torch.Generator("cpu").manual_seed(1)).to("cuda", DTYPE)
    slot = torch.tensor([2, 0], dtype=torch.int32, device="cuda")[:sequences]
    whole = block(u, slot)
    block.reset()
    parts = [block(u[:, :prompt].contiguous(), slot)]
    parts += [block(u[:, t:t + 1].contiguous(), slot) for t in range(prompt, prompt + tokens)]
    return whole, torch.cat(parts, 1)


if __name__ == "__main__":
    whole, parts = serve()
    off = (whole.double() - parts.double()).norm() / whole.double().norm()
    print(f"{tuple(whole.shape)} rows: prompt at once against prompt and single tokens, relative difference {off:.2e}")
