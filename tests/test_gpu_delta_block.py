"""The gated delta rule, the convolution before it, the normalisation behind it and the microscaled layers
around them, together as a block uses them (examples/delta_block.py)."""
import importlib.util
import os

import numpy as np
import pytest

import block_reference as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("delta_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_mix(block, p):
    """DeltaBlock.mix in 64 bits for one sequence p [length, columns]."""
    m, h, dk, dv, keys = block.mixed, block.heads, block.dk, block.dv, block.key_heads * block.dk
    p = p.double()
    taps = block.conv_w.shape[1]
    xx = torch.cat((p.new_zeros((taps - 1, m)), p[:, :m]))
    x = torch.nn.functional.silu(sum(xx[j:j + len(p)] * block.conv_w[:, j].double() for j in range(taps)))
    q, k = (x[:, i * keys:(i + 1) * keys].reshape(len(p), -1, dk) for i in range(2))
    q, k = ((t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(h // block.key_heads, 1) for t in (q, k))
    v, at = x[:, 2 * keys:].reshape(len(p), h, dv), m + h * dv
    decay = torch.exp(torch.nn.functional.softplus(p[:, at:at + h] + block.dt_bias.double()) * block.a.double())
    beta = torch.sigmoid(p[:, at + h:])
    S, out = p.new_zeros((h, dk, dv)), []
    for t in range(len(p)):
        S = decay[t][:, None, None] * S
        S = S + k[t][..., None] * (beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S)))[:, None]
        out.append(torch.einsum("hk,hkv->hv", q[t], S) * dk ** -0.5)
    y = torch.stack(out)
    y = (y / (y.square().mean(-1, keepdim=True) + 1e-5).sqrt()).flatten(1) * block.norm.double()
    return y * torch.nn.functional.silu(p[:, m:at])


@pytest.mark.parametrize("length", [1, 40, 130])
def test_mix_against_64_bits(example, length):
    """Three layers round to bf16: the convolution's outputs (queries, keys and values: three factors of what
    follows), the rule's and the norm's, 2^-8 each at most.  Independent but for their size they add to
    sqrt(5) 2^-8; the norm's factor, which is off as its row is, makes them twice that at most."""
    block = example.DeltaBlock()
    cols = block.in_proj.out
    p = torch.randn((2, length, cols), generator=torch.Generator("cpu").manual_seed(length)).to("cuda", torch.bfloat16)
    slot = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    prompt = block.mix(p, slot).view(2, length, -1)
    block.reset()
    tokens = torch.stack([block.mix(p[:, t:t + 1].contiguous(), slot) for t in range(length)], 1)
    for s in range(2):
        want = plain_mix(block, p[s])
        for got in (prompt, tokens):
            off = (got[s].double() - want).norm() / want.norm()
            assert off < 2 * 5 ** 0.5 * 2.0 ** -8, float(off)


@pytest.mark.parametrize("rows", [1, 30, 200])
def test_layer_is_the_product_of_what_was_quantised(example, rows):
    """Quantised rows times quantised weights: the definition's codes, and one rounding of a sum of 128 terms."""
    layer = example.Pointwise(torch.randn((96, 128), generator=torch.Generator("cpu").manual_seed(1)).to("cuda"))
    x = torch.randn((rows, 128), generator=torch.Generator("cpu").manual_seed(2)).to("cuda", torch.bfloat16)
    y = layer(x)
    widened = [ref.mx4_values(*ref.mx4_quantize(t.double().cpu().numpy())) for t in (x,)]
    w = ref.mx4_values(ref.unpack(layer.q.cpu().numpy()), layer.s.cpu().numpy().astype(np.int64))
    want, e = ref.mx4_matmul(widened[0], w, None, None, "none", "bf16")
    assert bool((np.abs(y.double().cpu().numpy() - want) <= e).all())


def test_prompt_and_tokens_agree(example):
    """A value whose neighbours differ by bf16's roundings (2^-8 a few times) crosses a border of the 4-bit grid (an
    eighth to a quarter of a value apart from the next) in one of some 16 cases, and is then a step off, a third at most:
    1/3 sqrt(1/16) = 1/12 of the layer's rows, which are themselves half of the block's result or less."""
    whole, parts = example.serve()
    off = (whole.double() - parts.double()).norm() / whole.double().norm()
    assert bool(torch.isfinite(whole).all()) and off < 1 / 12, float(off)


def test_block_in_a_graph(example):
    """The calls of a token, captured once and replayed, move the states on as the calls themselves."""
    u = torch.randn((6, 2, 1, 128), generator=torch.Generator("cpu").manual_seed(4)).to("cuda", torch.bfloat16)
    slot = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    block = example.DeltaBlock()
    want = [block(t, slot).clone() for t in u]
    states = block.state.clone(), block.conv_state.clone()
    token = u[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(token, slot)
    block.reset()
    for t, w in zip(u, want):
        token.copy_(t)
        graph.replay()
        assert bool((out == w).all())
    assert bool((block.state == states[0]).all()) and bool((block.conv_state == states[1]).all())
