"""The gated delta rule on the GPU against 64 bits, each element within the bound that the computation's own
roundings give (tests/block_reference.py)."""
import numpy as np
import pytest

import block_reference as ref
import pointwise_conv_cnn_gb300 as fcm
import seq_reference
from helpers import guarded_empty
from test_gpu_seq_layers import PACKED, beside, dev, ints, starts, within

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def run_delta(lengths, hk, heads, dk, dv, dtype, packed=True, seed=0, left=0, right=0, softplus=True, sigmoid=True,
              normalize=True, bias=True, scale=None, state_in=True, state_out=True, in_place=False, slots=None, slot=None,
              decay=1.0, alike=0.0, stream=None, max_len=None):
    """`alike`: how much the keys of a sequence are one key."""
    g = np.random.default_rng(seed)
    n_seq, tokens, at = len(lengths), sum(lengths), starts(lengths)
    slots = n_seq if slots is None else slots

    def rows(shape, x):
        cols = int(np.prod(shape))
        wide = g.standard_normal((tokens, left + cols + right))
        wide[:, left:left + cols] = x
        d, h = dev(wide, dtype)
        return d[:, left:left + cols].unflatten(1, shape), h[:, left:left + cols].reshape(tokens, *shape)
    keys = g.standard_normal((tokens, hk * dk)) * (1 - alike) + g.standard_normal(hk * dk) * alike
    if not normalize:   # of length one or so
        keys = keys / np.sqrt(dk)
    q, k = rows((hk, dk), g.standard_normal((tokens, hk * dk))), rows((hk, dk), keys)
    v = rows((heads, dv), g.standard_normal((tokens, heads * dv)))
    dt = rows((heads,), g.standard_normal((tokens, heads)) if softplus else -g.random((tokens, heads)))
    b = rows((heads,), g.standard_normal((tokens, heads)) if sigmoid else g.random((tokens, heads)))
    a = dev(g.uniform(0.2, 1.0, heads) * decay * (-1.0 if softplus else 1.0), "f32")
    bi = dev(g.uniform(-4.0, 0.0, heads), "f32") if bias and softplus else (None, None)
    old, old_h = dev(g.standard_normal((slots, heads, dk, dv)), "f32")
    y, unharmed = beside(tokens, heads * dv, dtype, left, right)
    out, guards = guarded_empty((slots, heads, dk, dv), "f32", fill=3.0)
    if in_place:
        out.copy_(old)
    f = (lambda t: t) if packed else (lambda t: t.unflatten(0, (n_seq, lengths[0])))
    where = dict(seq_start=ints(at), max_len=max(lengths) if max_len is None else max_len) if packed else {}
    fcm.gated_delta(f(q[0]), f(k[0]), f(v[0]), f(dt[0]), a[0], f(b[0]), f(y.unflatten(1, (heads, dv))), dt_bias=bi[0],
                    softplus=softplus, sigmoid=sigmoid, normalize=normalize, scale=scale, stream=stream,
                    slot=None if slot is None else ints(slot), state_in=(out if in_place else old) if state_in else None,
                    state_out=out if state_out else None, **where)
    torch.cuda.synchronize()
    unharmed(), guards()
    s32 = float(np.float32(dk ** -0.5 if scale is None else scale))
    want, e, state, e_state = ref.gated_delta(
        q[1], k[1], v[1], dt[1], a[1], b[1], bi[1], softplus, sigmoid, normalize, s32,
        seq_reference.bounds_of(n_seq, seq_start=at), slot, old_h if state_in else None, slots, dtype)
    within(y.unflatten(1, (heads, dv)), want, e, "y")
    mine = range(n_seq) if slot is None else slot
    for r in range(slots):
        if r in mine and state_out:
            within(out[r], state[r], np.broadcast_to(e_state[r], state[r].shape) + 1e-37, "state")
        else:
            assert bool((out[r] == (old[r] if in_place else 3.0)).all())
    return y, out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hk,heads,dk,dv", [(1, 2, 128, 128), (2, 2, 64, 32), (1, 3, 40, 33), (2, 4, 96, 80), (1, 1, 1, 1),
                                            (1, 1, 200, 48), (1, 2, 16, 8)])
@pytest.mark.parametrize("lengths", PACKED, ids=str)
def test_packed(lengths, hk, heads, dk, dv, dtype):
    run_delta(lengths, hk, heads, dk, dv, dtype, seed=dk + dv)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n_seq,length,heads,dk,dv", [(1, 1, 4, 128, 128), (70, 1, 2, 64, 64), (3, 41, 2, 128, 64),
                                                      (1, 300, 1, 128, 128), (2, 129, 2, 64, 100)])
@pytest.mark.parametrize("in_place", [False, True])
def test_equal_lengths(n_seq, length, heads, dk, dv, dtype, in_place):
    run_delta([length] * n_seq, heads, heads, dk, dv, dtype, packed=False, in_place=in_place, seed=length)


@pytest.mark.parametrize("softplus,sigmoid,normalize,bias", [(False, True, True, False), (True, False, True, True),
                                                             (True, True, False, False), (False, False, False, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_options(softplus, sigmoid, normalize, bias, dtype):
    run_delta([70, 0, 3], 1, 2, 64, 64, dtype, softplus=softplus, sigmoid=sigmoid, normalize=normalize, bias=bias, scale=0.7)


@pytest.mark.parametrize("state_in,state_out", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("length", [1, 100])
def test_without_states(state_in, state_out, length):
    run_delta([length, 2], 1, 2, 64, 64, "bf16", state_in=state_in, state_out=state_out)


@pytest.mark.parametrize("left,right", [(8, 8), (1, 0), (3, 4), (4, 4), (64, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_column_blocks(left, right, dtype):
    run_delta([70, 7], 1, 2, 64, 64, dtype, left=left, right=right)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slots(in_place, dtype):
    run_delta([65, 2, 0, 40], 1, 2, 64, 40, dtype, slots=9, slot=[7, -1, 3, 0], in_place=in_place)
    run_delta([1, 1, 1], 1, 2, 64, 40, dtype, packed=False, slots=4, slot=[2, 4, 1 << 30], in_place=in_place)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 30.0, 1e4, 1e30])
def test_decays(decay, dtype):
    """None at all, and ones that leave nothing: e^G is 1, tiny and 0."""
    run_delta([150], 1, 2, 64, 32, dtype, decay=decay)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("alike", [0.9, 1.0])
def test_keys_that_are_one_key(alike, dtype):
    """A chunk's triangular system is furthest from the unit matrix where its keys are the same."""
    run_delta([200], 1, 1, 64, 32, dtype, alike=alike, decay=0.01)


def test_loose_bounds_of_the_lengths():
    for max_len in (70, 71, 1000, 1 << 30):
        run_delta([70, 3], 1, 2, 64, 32, "bf16", max_len=max_len)


def test_bounds_outside_the_tokens():
    """seq_start past the rows, or before them, is cut; rows of no sequence are left."""
    q, v, dt = torch.ones(6, 1, 64, device="cuda"), torch.ones(6, 1, 32, device="cuda"), torch.zeros(6, 1, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((6, 1, 32), 7.0, device="cuda", dtype=dtype)
        fcm.gated_delta(q.to(dtype), q.to(dtype), v.to(dtype), dt.to(dtype), torch.zeros(1, device="cuda"), dt.to(dtype), y,
                        seq_start=ints([-5, 2, 1 << 30]), max_len=3)
        assert bool((y[5] == 7.0).all()) and bool((y[:5] != 7.0).all())


@pytest.mark.parametrize("length", [20, 130])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_stays_in_its_sequence_and_head(length, dtype):
    g = np.random.default_rng(5)
    t = 2 * length
    q, k, v = (dev(g.standard_normal((t, 2, 64)), dtype)[0] for _ in range(3))
    dt, b = (dev(g.standard_normal((t, 2)), dtype)[0] for _ in range(2))
    k[length - 1, 0, 3], v[length - 3, 0, 2], v[length - 2, 0, 5] = float("nan"), float("inf"), float("nan")
    y, out = torch.empty_like(v), torch.empty((2, 2, 64, 64), device="cuda")
    fcm.gated_delta(q, k, v, dt, -torch.ones(2, device="cuda"), b, y, seq_start=ints([0, length, t]), state_out=out)
    assert bool(torch.isfinite(y[:, 1]).all()) and bool(torch.isfinite(y[length:]).all())
    assert bool(torch.isnan(y[length - 1, 0]).all())
    assert bool(torch.isfinite(out[:, 1]).all()) and bool(torch.isfinite(out[1]).all()) and bool(torch.isnan(out[0, 0]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_bit_for_bit_on_streams_and_in_a_graph(dtype):
    g = np.random.default_rng(6)
    q, k, v = (dev(g.standard_normal((1, 200, 2, 64)), dtype)[0] for _ in range(3))
    dt, b = (dev(g.standard_normal((1, 200, 2)), dtype)[0] for _ in range(2))
    a, old = -torch.ones(2, device="cuda"), dev(g.standard_normal((1, 2, 64, 64)), "f32")[0]

    def call(stream=None):
        y, out = torch.empty_like(v), torch.empty_like(old)
        fcm.gated_delta(q, k, v, dt, a, b, y, state_in=old, state_out=out, stream=stream)
        return y, out
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [call(side), call(side.cuda_stream)]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(call())
    for t in got[-1]:
        t.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    for y, out in got:
        assert bool((y == want[0]).all()) and bool((out == want[1]).all())
