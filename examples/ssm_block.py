"""A gated state space block served with the framework's layers: a prompt at once, then token by
token from the states it left.

    xz        = in_proj(u)                                  pointwise  C -> 2D
    x         = silu(causal depthwise conv(xz[:, :D]))
    dt, B, C  = x_proj(x)                                   pointwise  D -> R + 2N
    delta     = dt_proj(dt)                                 pointwise  R -> D
    y         = selective scan(x, delta, a, B, C, skip, gate xz[:, D:])
    out       = u + out_proj(y)                             pointwise  D -> C

The pointwise layers' weights are 4-bit with group scales.  A prompt's rows go through the framework's
pointwise convolution on the same weights widened once; a few tokens' rows through the 4-bit
product, which reads a quarter of the bytes.  Convolution and scan take both, and hand their states
on in place.  Run: python examples/ssm_block.py"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import pointwise_conv_cnn_gb300 as fcm  # noqa: E402

DTYPE = torch.bfloat16
GROUP = 32
FEW = 16   # rows up to which the 4-bit product is used
LEAST, MOST = 64, 4096   # rows of the pointwise convolutions that a layer keeps: the powers of two between


def quantise(w: torch.Tensor):
    """w [out, in] -> (bytes [out, in / 2], scales [out, in / GROUP]): q = round(w / scale) + 8 in 0..15,
    an even column in a byte's low half."""
    o, k = w.shape
    g = w.view(o, k // GROUP, GROUP)
    scale = (g.abs().amax(-1) / 7.0).clamp_min(1e-8).to(DTYPE)
    q = (g / scale.float()[..., None]).round().clamp(-8, 7).to(torch.uint8).add(8).bitwise_and(15).view(o, k)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale


def widen(qw: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    q = torch.stack((qw & 15, qw >> 4), -1).flatten(1).float() - 8.0
    return (q * scale.float().repeat_interleave(GROUP, 1)).to(DTYPE)


class Pointwise:
    """y = x W^T on rows of tokens, W in 4 bits."""

    def __init__(self, w: torch.Tensor):
        self.qw, self.scale = (t.contiguous() for t in quantise(w))
        self.out, self.inp = w.shape
        self.modules = {}   # the pointwise convolution for each piece of a prompt

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        rows = x.shape[0]
        y = torch.empty((rows, self.out), dtype=DTYPE, device=x.device)
        if rows <= FEW:
            fcm.w4_matvec(x, self.qw, self.scale, y, GROUP)
            return y
        # A convolution is planned for its rows.  A prompt goes through in pieces of powers of two, the last one
        # filled up, so that a layer keeps a handful of them whatever lengths it meets.
        x, at = x.contiguous(), 0
        while rows - at >= LEAST:
            n = min(MOST, 1 << ((rows - at).bit_length() - 1))
            self.module(n).run(x[at:at + n], y[at:at + n], "pw")
            at += n
        if at < rows:
            piece = torch.zeros((LEAST, self.inp), dtype=DTYPE, device=x.device)
            piece[:rows - at] = x[at:]
            out = torch.empty((LEAST, self.out), dtype=DTYPE, device=x.device)
            self.module(LEAST).run(piece, out, "pw")
            y[at:] = out[:rows - at]
        return y

    def module(self, rows: int) -> fcm.FusedConvModule:
        if rows not in self.modules:
            one, zero = torch.ones(max(self.out, self.inp)), torch.zeros(max(self.out, self.inp))
            desc = fcm.make_desc(n=1, h=1, w=rows, c=self.inp, k_out=self.out, ksize=1, stride=1, pad=0,
                                 conv1="dw", dtype="bf16", act1="none", act2="none")
            self.modules[rows] = fcm.FusedConvModule(
                desc, torch.ones(self.inp, dtype=DTYPE), widen(self.qw, self.scale).cpu(), one, zero, one, zero)
        return self.modules[rows]


class SsmBlock:
    """One block with its states; `slots` sequences can be in flight."""

    def __init__(self, c=128, d=256, n=16, r=32, k=4, slots=4, seed=0, device="cuda"):
        g = torch.Generator("cpu").manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(device)
        self.d, self.n, self.r = d, n, r
        self.in_proj, self.x_proj = Pointwise(normal(2 * d, c)), Pointwise(normal(r + 2 * n, d))
        self.dt_proj, self.out_proj = Pointwise(normal(d, r)), Pointwise(normal(c, d))
        self.conv_w, self.conv_b = normal(d, k).to(DTYPE), 0.1 * torch.randn(d, generator=g).to(device)
        self.a = -torch.arange(1, n + 1, dtype=torch.float32, device=device).repeat(d, 1)
        self.skip = torch.ones(d, device=device)
        self.dt_bias = torch.linspace(-6.0, -2.0, d, device=device)
        self.conv_state = torch.zeros((slots, k - 1, d), dtype=DTYPE, device=device)
        self.scan_state = torch.zeros((slots, d, n), device=device)

    def __call__(self, u: torch.Tensor, slot: torch.Tensor) -> torch.Tensor:
        """u [sequences, length, c]: the next rows of the sequences whose states are in rows `slot`
        (int32 [sequences]); the states move on."""
        s, length, c = u.shape
        xz = self.in_proj(u.reshape(-1, c)).view(s, length, -1)
        x = torch.empty((s, length, self.d), dtype=DTYPE, device=u.device)
        fcm.causal_conv(xz[..., :self.d], self.conv_w, x, bias=self.conv_b, act="silu", slot=slot,
                        state_in=self.conv_state, state_out=self.conv_state)
        proj = self.x_proj(x.view(-1, self.d))
        delta = self.dt_proj(proj[:, :self.r]).view(s, length, self.d)
        b, cc = (proj[:, at:at + self.n].view(s, length, self.n) for at in (self.r, self.r + self.n))
        y = torch.empty_like(x)
        fcm.selective_scan(x, delta, self.a, b, cc, y, skip=self.skip, z=xz[..., self.d:],
                           dt_bias=self.dt_bias, slot=slot, state_in=self.scan_state, state_out=self.scan_state)
        return u + self.out_proj(y.view(-1, self.d)).view(s, length, c)

    def reset(self) -> None:
        self.conv_state.zero_()
        self.scan_state.zero_()


def serve(prompt=50, tokens=12, sequences=2, c=128) -> tuple[torch.Tensor, torch.Tensor]:
    """The same rows once as one prompt, once as a shorter prompt and single tokens."""
    block = SsmBlock(c=c)
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
