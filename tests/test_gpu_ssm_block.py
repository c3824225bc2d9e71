"""The example that serves a state space block with the framework's layers (examples/ssm_block.py)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ssm_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("ssm_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(block, u):
    """The block in 64 bits on the example's weights, one sequence u [length, c]."""
    w = {k: _wide(getattr(block, k)) for k in ("in_proj", "x_proj", "dt_proj", "out_proj")}
    d, n, r = block.d, block.n, block.r
    u = u.double()
    xz = u @ w["in_proj"].T
    k = block.conv_w.shape[1]
    xx = torch.cat((u.new_zeros((k - 1, d)), xz[:, :d]))
    x = torch.nn.functional.silu(sum(xx[j:j + len(u)] * block.conv_w[:, j].double() for j in range(k)) + block.conv_b)
    proj = x @ w["x_proj"].T
    delta = torch.nn.functional.softplus(proj[:, :r] @ w["dt_proj"].T + block.dt_bias)
    h, out = u.new_zeros((d, n)), []
    for t in range(len(u)):
        h = torch.exp(delta[t][:, None] * block.a) * h + (delta[t] * x[t])[:, None] * proj[t, r:r + n]
        out.append(h @ proj[t, r + n:] + block.skip * x[t])
    y = torch.stack(out) * torch.nn.functional.silu(xz[:, d:])
    return u + y @ w["out_proj"].T


def _wide(layer):
    q = torch.stack((layer.qw & 15, layer.qw >> 4), -1).flatten(1).double() - 8.0
    return q * layer.scale.double().repeat_interleave(q.shape[1] // layer.scale.shape[1], 1)


def test_block_against_64_bits(example):
    """Ten roundings to bf16 (five layers' outputs, their weights' widening, the sum) at 2^-8 each at
    most, of values that the block's layers keep at the size of its rows: 2^-8 * sqrt(10) if they
    are independent, which they are but for their size."""
    block = example.SsmBlock()
    u = torch.randn((2, 40, 128), generator=torch.Generator("cpu").manual_seed(3)).to("cuda", torch.bfloat16)
    slot = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    prompt = block(u, slot)
    block.reset()
    tokens = torch.cat([block(u[:, t:t + 1].contiguous(), slot) for t in range(40)], 1)
    for s in range(2):
        want = plain(block, u[s])
        for got in (prompt, tokens):
            off = (got[s].double() - want).norm() / want.norm()
            assert off < 2.0 ** -8 * 10 ** 0.5, float(off)


def test_prompt_and_tokens_agree(example):
    whole, parts = example.serve()
    off = (whole.double() - parts.double()).norm() / whole.double().norm()
    assert off < 2 * 2.0 ** -8 * 10 ** 0.5, float(off)
