"""The gated delta rule with states that grow, steadily and between decays, in both of its kernels, against 64 bits
with the bound that the computation's own roundings give (tests/block_reference.py)."""
import numpy as np
import pytest

import block_reference as ref
import pointwise_conv_cnn_gb300 as fcm
import seq_reference
from launches import launch_of
from test_gpu_seq_layers import dev, ints, starts, within

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def dip(n):
    G = np.zeros(n)
    G[n // 4], G[n // 2] = -20.0, 20.0
    return G


# The logarithms of a sequence's factors, row by row; their sum stays below 88, a float's range.
GROWTH = {
    "0.1": lambda n: np.full(n, 0.1), "0.5": lambda n: np.full(n, 0.5), "2": lambda n: np.full(n, 2.0),
    "5, -5": lambda n: np.resize([5.0, -5.0], n), "-5, 5": lambda n: np.resize([-5.0, 5.0], n),
    "30, -30": lambda n: np.resize([30.0, -30.0], n), "-20 .. 20": dip,
    "up and down": lambda n: np.where(np.arange(n) < n // 2, 2.0, -2.0),
    "down and up": lambda n: np.where(np.arange(n) < n // 2, -2.0, 2.0),
    "any": lambda n: np.random.default_rng(4).normal(0.0, 3.0, n).clip(-8.0, 8.0),
}


def run(lengths, G, dtype, dk, dv=40, heads=2, softplus=False, seed=0, max_len=None):
    """G [tokens, heads]; queries are scaled by what the largest state has grown, so that y fits its type."""
    g = np.random.default_rng(seed)
    tokens, at = sum(lengths), starts(lengths)
    q, k, v = (dev(g.standard_normal((tokens, heads, c)), dtype) for c in (dk, dk, dv))
    b = dev(g.standard_normal((tokens, heads)), dtype)
    dt = dev(np.log(np.expm1(G)) if softplus else G, dtype)
    a = dev(np.ones(heads), "f32")
    most = max(np.maximum.accumulate(G[s:e].cumsum(0)).max() for s, e in zip(at, at[1:]))
    scale = float(np.float32(np.exp(-max(most, 0.0)) * dk ** -0.5))
    old, old_h = dev(g.standard_normal((len(lengths), heads, dk, dv)), "f32")
    y, out = torch.empty_like(v[0]), torch.empty_like(old)

    def call(stream=None):
        fcm.gated_delta(q[0], k[0], v[0], dt[0], a[0], b[0], y, softplus=softplus, scale=scale, seq_start=ints(at),
                        max_len=max(lengths) if max_len is None else max_len, state_in=old, state_out=out, stream=stream)
    call()
    want, e, state, e_state = ref.gated_delta(
        q[1], k[1], v[1], dt[1], a[1], b[1], None, softplus, True, True, scale,
        seq_reference.bounds_of(len(lengths), seq_start=at), None, old_h, len(lengths), dtype)
    assert np.isfinite(want).all() and np.isfinite(state).all() and np.abs(state).max() < 3e38
    got = y
    if dtype == "f16":   # from 65520 on a result rounds to infinity, up to 65504 it stays a number
        size = np.abs(want)
        got = y.double().cpu().numpy()
        past, sure = size + e >= 65504.0, size - e > 65520.0
        assert (got[sure] == np.sign(want[sure]) * np.inf).all()
        got = torch.from_numpy(np.where(past, want, got))
    within(got, want, e, "y")
    within(out, state, np.broadcast_to(e_state, state.shape), "state")
    return call


@pytest.mark.parametrize("dtype,dk,lengths,kernel", [
    ("f32", 64, [40, 3], "delta_row"), ("bf16", 128, [15, 14], "delta_row"), ("f16", 200, [40], "delta_row"),
    ("bf16", 64, [40, 33, 3], "delta_chunk"), ("bf16", 128, [32, 16], "delta_chunk"), ("f16", 64, [31, 40], "delta_chunk"),
    ("f16", 128, [40], "delta_chunk")])
@pytest.mark.parametrize("growth", GROWTH)
def test_growing_states(growth, dtype, dk, lengths, kernel):
    G = np.concatenate([GROWTH[growth](n) for n in lengths])
    call = run(lengths, np.stack([G, -0.25 * G], 1), dtype, dk)   # another head goes the other way
    assert kernel in launch_of(call).name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growth_through_softplus(dtype):
    run([36, 2], np.random.default_rng(5).uniform(0.3, 1.8, (38, 2)), dtype, 64, softplus=True)


@pytest.mark.parametrize("growth", ["0.5", "any"])
def test_short_sequences_with_any_bound_of_their_lengths(growth):
    """A row a sequence and a few, by the kernel of single tokens, of few rows, and in chunks."""
    G = np.concatenate([GROWTH[growth](n) for n in (1, 2, 1, 15)])
    for max_len in (15, 16, 1 << 20):
        run([1, 2, 1, 15], np.stack([G, G[::-1]], 1), "bf16", 64, max_len=max_len)


@pytest.mark.parametrize("dtype,dk", [("f32", 64), ("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("factor", [-2.0, -3.0, 3.0])
def test_keys_and_steps_that_multiply(factor, dtype, dk):
    """One key that is not of length 1: each row multiplies what is stored under it by 1 - B |k|^2, with no decay."""
    g = np.random.default_rng(7)
    tokens, heads, dv = 36, 2, 40
    key = g.standard_normal((heads, dk))
    key *= 2.0 / np.sqrt((key * key).sum(-1, keepdims=True))
    k = dev(np.repeat(key[None], tokens, 0), dtype)
    b = dev(np.full((tokens, heads), (1.0 - factor) / 4.0), dtype)
    q, v = (dev(g.standard_normal((tokens, heads, c)), dtype) for c in (dk, dv))
    dt, a = dev(np.zeros((tokens, heads)), dtype), dev(np.ones(heads), "f32")
    scale = float(np.float32(abs(factor) ** -tokens))
    y, out = torch.empty_like(v[0]), torch.empty((1, heads, dk, dv), device="cuda")
    fcm.gated_delta(q[0], k[0], v[0], dt[0], a[0], b[0], y, softplus=False, sigmoid=False, normalize=False, scale=scale,
                    seq_start=ints([0, tokens]), max_len=tokens, state_out=out)
    want, e, state, e_state = ref.gated_delta(q[1], k[1], v[1], dt[1], a[1], b[1], None, False, False, False, scale,
                                              [(0, tokens)], None, None, 1, dtype)
    within(y, want, e, "y")
    within(out, state, np.broadcast_to(e_state, state.shape), "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("length", [20, 100])
def test_infinite_growth_stays_visible(dtype, length):
    """From an infinite factor on nothing of that head looks like a number; the other head and sequence do not notice."""
    g = np.random.default_rng(6)
    q, k, v = (dev(g.standard_normal((2 * length, 2, 64)), dtype)[0] for _ in range(3))
    dt, b = (dev(g.uniform(-1.0, 0.0, (2 * length, 2)), dtype)[0] for _ in range(2))
    dt[length - 5, 0], dt[length - 3, 0] = float("inf"), -2000.0
    y, out = torch.empty_like(v), torch.empty((2, 2, 64, 64), device="cuda")
    fcm.gated_delta(q, k, v, dt, torch.ones(2, device="cuda"), b, y, softplus=False, seq_start=ints([0, length, 2 * length]),
                    state_out=out)
    assert not bool(torch.isfinite(y[length - 5:length, 0]).any()) and not bool(torch.isfinite(out[0, 0]).any())
    assert bool(torch.isfinite(y[:, 1]).all()) and bool(torch.isfinite(y[length:]).all())
    assert bool(torch.isfinite(out[:, 1]).all()) and bool(torch.isfinite(out[1]).all())
