"""The layers over sequences on the GPU against the 64-bit references, each element within the bound
that the computation's own roundings give (tests/seq_reference.py)."""
import numpy as np
import pytest

import pointwise_conv_cnn_gb300 as fcm
import seq_reference as ref
from helpers import guarded_empty, torch_dtype

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def dev(a, dtype):
    """The array rounded to the storage type on the GPU, and the rounded values in 64 bits."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(torch_dtype(dtype)).cuda()
    return t, t.double().cpu().numpy()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def within(got, want, bound, what):
    got = got.double().cpu().numpy()
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {want[bad][0]}, "
                           f"bound {bound[bad][0]:.3g}")


def beside(rows, cols, dtype, left, right):
    """A column block [left : left + cols] of a wider tensor, and a check of its neighbours."""
    wide, check = guarded_empty((rows, left + cols + right), dtype, fill=7.0)

    def unharmed():
        check()
        assert bool((wide[:, :left] == 7.0).all()) and bool((wide[:, left + cols:] == 7.0).all())
    return wide[:, left:left + cols], unharmed


# Packed sequences: lengths from none to past every tile.
PACKED = [[5], [1], [0], [1, 1, 1], [3, 0, 1, 70], [0, 0, 130, 2, 17], [33, 64, 16, 15, 0, 1]]


def starts(lengths):
    return [sum(lengths[:i]) for i in range(len(lengths) + 1)]


def run_conv(lengths, c, k, dtype, act="silu", packed=True, seed=0, left=0, right=0, scale=True,
             bias=True, state_in=True, in_place=False, slots=None, slot=None, x=None):
    g = np.random.default_rng(seed)
    n_seq, tokens, at = len(lengths), sum(lengths), starts(lengths)
    slots = n_seq if slots is None else slots
    xd, xh = dev(g.standard_normal((tokens, left + c + right)) if x is None else x, dtype)
    xd, xh = xd[:, left:left + c], xh[:, left:left + c]
    wd, wh = dev(g.standard_normal((c, k)) / np.sqrt(k), dtype)
    sd, sh = dev(g.uniform(0.5, 1.5, c), "f32") if scale else (None, None)
    bd, bh = dev(g.standard_normal(c), "f32") if bias else (None, None)
    old, old_h = dev(g.standard_normal((slots, k - 1, c)), dtype)
    y, unharmed = beside(tokens, c, dtype, left, right)
    out, guards = guarded_empty((slots, k - 1, c), dtype, fill=3.0)
    if in_place:
        out.copy_(old)
    kw = dict(scale=sd, bias=bd, act=act, slot=None if slot is None else ints(slot), state_out=out,
              state_in=(out if in_place else old) if state_in else None)
    if packed:
        fcm.causal_conv(xd, wd, y, seq_start=ints(at), max_len=max(lengths), **kw)
    else:
        fcm.causal_conv(xd.unflatten(0, (n_seq, lengths[0])), wd,
                        y.unflatten(0, (n_seq, lengths[0])), **kw)
    torch.cuda.synchronize()
    unharmed(), guards()
    want, e, state = ref.causal_conv(xh, wh, sh, bh, act, ref.bounds_of(n_seq, seq_start=at), slot,
                                     old_h if state_in else None, slots, dtype)
    within(y, want, e, "y")
    rows = range(n_seq) if slot is None else slot
    for r in range(slots):
        if r in rows:
            np.testing.assert_array_equal(out[r].double().cpu().numpy(), state[r])
        else:   # a row of no sequence keeps what it held
            assert bool((out[r] == (old[r] if in_place else 3.0)).all())
    return y, out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c,k", [(64, 4), (40, 3), (37, 4), (1, 2), (8, 8), (130, 5), (16, 1)])
@pytest.mark.parametrize("lengths", PACKED, ids=str)
def test_conv_packed(lengths, c, k, dtype):
    if sum(lengths) == 0 and k == 1:
        pytest.skip("nothing to compute or keep")
    run_conv(lengths, c, k, dtype, seed=c + k)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n_seq,length,c", [(1, 1, 72), (5, 1, 72), (300, 1, 33), (3, 41, 24), (1, 500, 264)])
@pytest.mark.parametrize("in_place", [False, True])
def test_conv_equal_lengths(n_seq, length, c, dtype, in_place):
    run_conv([length] * n_seq, c, 4, dtype, packed=False, in_place=in_place, seed=length)


@pytest.mark.parametrize("act", ["none", "relu", "relu6", "silu"])
@pytest.mark.parametrize("scale,bias,state_in", [(False, False, False), (True, False, True), (False, True, True)])
def test_conv_options(act, scale, bias, state_in):
    run_conv([6, 0, 3], 24, 4, "f16", act=act, scale=scale, bias=bias, state_in=state_in)


@pytest.mark.parametrize("left,right", [(8, 8), (64, 0), (1, 0), (0, 1), (3, 4), (4, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_column_blocks(left, right, dtype):
    run_conv([20, 7], 64, 4, dtype, left=left, right=right)


@pytest.mark.parametrize("in_place", [False, True])
def test_conv_slots(in_place):
    """States anywhere in a larger pool; sequences without a slot start from zero."""
    run_conv([5, 2, 0, 40], 48, 4, "bf16", slots=9, slot=[7, -1, 3, 0], in_place=in_place)
    run_conv([1, 1, 1], 48, 4, "bf16", packed=False, slots=4, slot=[2, 4, 1 << 30], in_place=in_place)


def test_conv_infinities_stay_in_their_sequence():
    x = np.random.default_rng(3).standard_normal((30, 16))
    x[9], x[10, 3] = np.nan, np.inf          # the last rows of the first sequence
    g = np.random.default_rng(4)
    wd, _ = dev(np.abs(g.standard_normal((16, 3))), "f32")
    xd, _ = dev(x, "f32")
    y = torch.empty_like(xd)
    out = torch.empty((2, 2, 16), device="cuda")
    fcm.causal_conv(xd, wd, y, act="none", seq_start=ints([0, 11, 30]), state_out=out)
    assert bool(torch.isfinite(y[:9]).all()) and bool(torch.isfinite(y[11:]).all())
    assert bool(torch.isnan(y[9:11]).all())
    assert bool(torch.isfinite(out[1]).all()) and bool(torch.isnan(out[0, 0]).all())


# ------------------------------------------------------------------------------ selective scan
def scan_inputs(g, tokens, c, n, groups, dtype, left=0, right=0, z=True):
    def rows(cols, std=1.0):
        d, h = dev(g.standard_normal((tokens, left + cols + right)) * std, dtype)
        return d[:, left:left + cols], h[:, left:left + cols]
    x, dt = rows(c), rows(c, 1.0)
    bm, cm = (tuple(v.reshape(tokens, groups, n) if isinstance(v, np.ndarray) else v.unflatten(1, (groups, n))
                    for v in rows(groups * n)) for _ in range(2))
    a = dev(-np.exp(g.uniform(np.log(0.2), np.log(16.0), (c, n))), "f32")
    skip, bias = dev(g.standard_normal(c), "f32"), dev(g.uniform(-5.0, 0.0, c), "f32")
    return x, dt, a, bm, cm, skip, (rows(c) if z else (None, None)), bias


def run_scan(lengths, c, n, dtype, groups=1, packed=True, seed=0, left=0, right=0, z=True, skip=True,
             bias=True, softplus=True, state_in=True, in_place=False, slots=None, slot=None):
    g = np.random.default_rng(seed)
    n_seq, tokens, at = len(lengths), sum(lengths), starts(lengths)
    slots = n_seq if slots is None else slots
    x, dt, a, bm, cm, sk, zz, bi = scan_inputs(g, tokens, c, n, groups, dtype, left, right, z)
    if not softplus:   # steps as they are used: positive, and some of none
        dt = dev(np.abs(dt[1]) * 0.3 * (g.random((tokens, c)) > 0.1), dtype)
    sk = sk if skip else (None, None)
    bi = bi if bias and softplus else (None, None)
    old, old_h = dev(g.standard_normal((slots, c, n)), "f32")
    y, unharmed = beside(tokens, c, dtype, left, right)
    out, guards = guarded_empty((slots, c, n), "f32", fill=3.0)
    if in_place:
        out.copy_(old)
    kw = dict(skip=sk[0], dt_bias=bi[0], softplus=softplus, state_out=out,
              slot=None if slot is None else ints(slot),
              state_in=(out if in_place else old) if state_in else None)
    if packed:
        fcm.selective_scan(x[0], dt[0], a[0], bm[0], cm[0], y, z=zz[0], seq_start=ints(at),
                           max_len=max(lengths), **kw)
    else:
        f = lambda t: None if t is None else t.unflatten(0, (n_seq, lengths[0]))  # noqa: E731
        fcm.selective_scan(f(x[0]), f(dt[0]), a[0], f(bm[0]), f(cm[0]), f(y), z=f(zz[0]), **kw)
    torch.cuda.synchronize()
    unharmed(), guards()
    want, e, state, e_state = ref.selective_scan(
        x[1], dt[1], a[1], bm[1], cm[1], sk[1], zz[1], bi[1], softplus,
        ref.bounds_of(n_seq, seq_start=at), slot, old_h if state_in else None, slots, dtype)
    within(y, want, e, "y")
    rows = range(n_seq) if slot is None else slot
    for r in range(slots):
        if r in rows:
            within(out[r], state[r], e_state[r] + 1e-37, "state")
        else:
            assert bool((out[r] == (old[r] if in_place else 3.0)).all())
    return y, out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c,n,groups", [(64, 16, 1), (37, 16, 1), (40, 8, 2), (1, 1, 1), (6, 3, 2),
                                        (24, 64, 3), (34, 12, 1), (5, 128, 1), (32, 4, 1), (9, 33, 1)])
@pytest.mark.parametrize("lengths", PACKED, ids=str)
def test_scan_packed(lengths, c, n, groups, dtype):
    run_scan(lengths, c, n, dtype, groups, seed=c + n)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n_seq,length,c,n", [(1, 1, 72, 16), (5, 1, 40, 16), (200, 1, 33, 5),
                                              (3, 41, 24, 16), (1, 1100, 40, 16), (2, 300, 264, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_scan_equal_lengths(n_seq, length, c, n, dtype, in_place):
    run_scan([length] * n_seq, c, n, dtype, packed=False, in_place=in_place, seed=length)


@pytest.mark.parametrize("kw", [dict(z=False), dict(skip=False), dict(bias=False), dict(softplus=False),
                                dict(state_in=False), dict(z=False, skip=False, bias=False)], ids=str)
@pytest.mark.parametrize("lengths", [[1, 1, 1], [9, 0, 50]], ids=str)
def test_scan_options(lengths, kw):
    run_scan(lengths, 40, 16, "f16", packed=len(set(lengths)) > 1, **kw)


@pytest.mark.parametrize("left,right", [(8, 8), (64, 0), (1, 0), (0, 1), (3, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[20, 70], [1, 1]], ids=str)
def test_scan_column_blocks(lengths, left, right, dtype):
    run_scan(lengths, 64, 16, dtype, left=left, right=right)


@pytest.mark.parametrize("in_place", [False, True])
def test_scan_slots(in_place):
    run_scan([5, 2, 0, 40], 48, 16, "bf16", slots=9, slot=[7, -1, 3, 0], in_place=in_place)
    run_scan([1, 1, 1], 48, 16, "bf16", packed=False, slots=4, slot=[2, 4, 1 << 30], in_place=in_place)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c,n,groups", [(64, 12, 1), (40, 20, 1), (45, 28, 1), (24, 40, 1), (17, 42, 1),
                                        (16, 72, 1), (10, 76, 2), (128, 12, 2), (126, 16, 1)])
@pytest.mark.parametrize("left,right", [(0, 0), (3, 0)])
def test_scan_odd_states_and_rows(c, n, groups, left, right, dtype):
    """State counts that leave lanes of a channel empty, or part of one; rows of the channels and
    of the states that start on 16 bytes or do not, each with the other."""
    run_scan([33, 0, 70], c, n, dtype, groups, left=left, right=right, seed=c + n)


@pytest.mark.parametrize("n", [12, 20, 40])
def test_scan_infinities_and_empty_lanes(n):
    """What an infinite input makes of the states that there are does not meet those that there are not."""
    c, length = 20, 40
    x = torch.ones((1, length, c), device="cuda")
    x[0, 5, 3] = float("inf")
    one = torch.ones((1, length, n), device="cuda")
    y = torch.empty_like(x)
    fcm.selective_scan(x, torch.ones_like(x), -0.01 * torch.ones((c, n), device="cuda"), one, one, y,
                       softplus=False)
    assert bool((y[0, 5:, 3] == float("inf")).all()) and bool(torch.isfinite(y[0, :5]).all())
    y[0, :, 3] = 0
    assert bool(torch.isfinite(y).all())


@pytest.mark.parametrize("n", [1, 3, 5, 16])
@pytest.mark.parametrize("length", [1, 40])
def test_scan_infinities_stay_where_they_are(n, length):
    """An infinite input drives its own channel's states to infinity with B's signs, and no other
    channel, whatever the state count is rounded up to inside."""
    c = 20
    x = torch.ones((2, length, c), device="cuda")
    x[0, 0, 3] = float("inf")
    bm = torch.ones((2, length, n), device="cuda")
    y = torch.empty_like(x)
    out = torch.empty((2, c, n), device="cuda")
    fcm.selective_scan(x, torch.ones_like(x), -0.01 * torch.ones((c, n), device="cuda"), bm, bm, y,
                       softplus=False, state_out=out)
    assert bool((y[0, :, 3] == float("inf")).all()) and bool((out[0, 3] == float("inf")).all())
    rest = torch.ones((2, c), dtype=torch.bool, device="cuda")
    rest[0, 3] = False
    assert bool(torch.isfinite(y.transpose(1, 2)[rest]).all()) and bool(torch.isfinite(out[rest]).all())


def test_scan_extreme_steps():
    """Steps of 0 keep the state, steps far above what softplus changes pass through, decays that
    reach 0 forget it; pre-softplus values of minus infinity are steps of 0."""
    c, n, length = 12, 4, 6
    x = torch.ones((1, length, c), device="cuda")
    dt = torch.zeros((1, length, c), device="cuda")
    dt[..., 0] = float("-inf")
    dt[..., 1] = 100.0
    dt[..., 2] = -100.0
    one = torch.ones((1, length, n), device="cuda")
    a = -torch.ones((c, n), device="cuda")
    old = torch.full((1, c, n), 2.0, device="cuda")
    out = torch.empty_like(old)
    y = torch.empty_like(x)
    fcm.selective_scan(x, dt, a, one, one, y, state_in=old, state_out=out)
    assert bool((out[0, 0] == 2.0).all()) and bool((y[0, :, 0] == 2.0 * n).all())
    torch.testing.assert_close(out[0, 1], torch.full((n,), 100.0, device="cuda"), rtol=1e-6, atol=0)
    torch.testing.assert_close(out[0, 2], torch.full((n,), 2.0, device="cuda"), rtol=1e-6, atol=0)


@pytest.mark.parametrize("layer", ["conv", "scan"])
@pytest.mark.parametrize("cuts", [[64], [1] * 12, [3, 50, 1, 90]], ids=str)
def test_prompts_in_parts(layer, cuts):
    """A prompt in parts, the state handed on, against the prompt at once."""
    total, c, n = sum(cuts), 40, 16
    g = np.random.default_rng(5)
    x, dt, a, bm, cm, sk, zz, bi = scan_inputs(g, total, c, n, 1, "f32")
    w, wh = dev(g.standard_normal((c, 4)), "f32")
    y = torch.empty((total, c), device="cuda")
    state = torch.zeros((1, 3, c) if layer == "conv" else (1, c, n), device="cuda")
    at = 0
    for cut in cuts:
        p = slice(at, at + cut)
        if layer == "conv":
            fcm.causal_conv(x[0][None, p], w, y[None, p], state_in=state, state_out=state)
        else:
            fcm.selective_scan(x[0][None, p], dt[0][None, p], a[0], bm[0][None, p], cm[0][None, p],
                               y[None, p], skip=sk[0], z=zz[0][None, p], dt_bias=bi[0],
                               state_in=state, state_out=state)
        at += cut
    seqs = [(0, total)]
    if layer == "conv":
        want, e, last = ref.causal_conv(x[1], wh, None, None, "silu", seqs, None, None, 1, "f32")
        np.testing.assert_array_equal(state.cpu().numpy(), last.astype(np.float32))
    else:
        want, e, last, e_last = ref.selective_scan(x[1], dt[1], a[1], bm[1], cm[1], sk[1], zz[1],
                                                   bi[1], True, seqs, None, None, 1, "f32")
        within(state, last, e_last, "state")
    within(y, want, e, "y")


def test_bounds_that_lead_nowhere_are_cut():
    """seq_start is device memory: what lies outside the rows, or past max_len, is not touched."""
    c = 24
    for layer in ("conv", "scan"):
        y, guards = guarded_empty((10, c), "f32", fill=7.0)
        x = torch.ones((10, c), device="cuda")
        seq = ints([-5, 3, 2, 8, 1 << 30])     # -5..3 -> 0..3, 3..2 -> none, 2..8 -> 2..6, 8.. -> 8..10
        kw = dict(seq_start=seq, max_len=4)
        if layer == "conv":
            w = torch.ones((c, 4), device="cuda")
            fcm.causal_conv(x, w, y, act="none", **kw)
        else:
            one = torch.ones((10, 4), device="cuda")
            fcm.selective_scan(x, x, torch.zeros((c, 4), device="cuda"), one, one, y, softplus=False, **kw)
        torch.cuda.synchronize()
        guards()
        # rows 2 is written by two sequences here; 6 and 7 by none
        assert bool((y[6:8] == 7.0).all()) and bool((y[8] == (1.0 if layer == "conv" else 4.0)).all())
        assert bool((y[3:6, 0] != 7.0).all()) and bool((y[:2, 0] != 7.0).all())


# ------------------------------------------------------------------------------ 4-bit weights
def run_w4(m, o, k, group, dtype, act="none", fold=True, left=0, right=0, seed=0):
    g = np.random.default_rng(seed)
    xd, xh = dev(g.standard_normal((m, left + k + right)), dtype)
    q = g.integers(0, 16, (o, k))
    qs, qsh = dev(g.uniform(0.5, 1.5, (o, -(-k // group))) / np.sqrt(k), dtype)
    sd, sh = dev(g.uniform(0.5, 1.5, o), "f32") if fold else (None, None)
    bd, bh = dev(g.standard_normal(o), "f32") if fold else (None, None)
    y, unharmed = beside(m, o, dtype, left, right)
    fcm.w4_matvec(xd[:, left:left + k], torch.from_numpy(ref.pack_w4(q)).cuda(), qs, y, group,
                  scale=sd, bias=bd, act=act)
    torch.cuda.synchronize()
    unharmed()
    want, e = ref.w4_matvec(xh[:, left:left + k], q, qsh, group, sh, bh, act, dtype)
    within(y, want, e, "y")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,o,k", [(1, 1, 32), (1, 64, 128), (1, 77, 4096), (2, 33, 160), (3, 16, 96),
                                   (8, 130, 1024), (9, 15, 2080), (16, 48, 512), (17, 20, 320), (40, 9, 64),
                                   (1, 300, 8224), (5, 1030, 256)])
def test_w4(m, o, k, group, dtype):
    run_w4(m, o, k, group, dtype, seed=m + o)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,o,k,group", [(1, 2435, 4096, 128), (8, 2435, 4096, 128), (5, 4900, 4224, 128),
                                         (7, 2435, 4064, 128), (9, 2435, 2048, 64), (16, 2435, 4096, 128),
                                         (12, 4900, 4160, 64), (33, 1217, 4000, 128), (41, 833, 2080, 64)])
def test_w4_two_tiles_of_outputs(m, o, k, group, dtype):
    """Enough outputs and inputs for blocks of 32 outputs, with a last block, a last token and a last
    group that are not whole, and scales that can and cannot be read four at a time."""
    run_w4(m, o, k, group, dtype, seed=m + o)


@pytest.mark.parametrize("act", ["none", "relu", "relu6", "silu"])
@pytest.mark.parametrize("fold", [False, True])
def test_w4_options(act, fold):
    run_w4(3, 40, 256, 64, "bf16", act=act, fold=fold)


@pytest.mark.parametrize("left,right", [(8, 8), (64, 0), (1, 0), (0, 1), (3, 4)])
def test_w4_column_blocks(left, right):
    run_w4(4, 40, 256, 128, "f16", left=left, right=right)


def test_w4_exact_on_small_integers():
    """Products and sums of small integers are exact in 32 bits, whatever the order."""
    g = np.random.default_rng(7)
    x, q = g.integers(-8, 9, (6, 512)).astype(np.float64), g.integers(0, 16, (50, 512))
    xd, _ = dev(x, "f16")
    qs = torch.ones((50, 4), dtype=torch.float16, device="cuda")
    y = torch.empty((6, 50), dtype=torch.float16, device="cuda")
    fcm.w4_matvec(xd, torch.from_numpy(ref.pack_w4(q)).cuda(), qs, y, 128)
    want = torch.from_numpy(x @ (q - 8.0).T).half()
    assert bool((y.cpu() == want).all())


def test_w4_infinities_stay_in_their_token():
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    x[1, 5] = float("nan")
    qw = torch.full((20, 32), 0x99, dtype=torch.uint8, device="cuda")
    qs = torch.ones((20, 2), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((3, 20), dtype=torch.bfloat16, device="cuda")
    fcm.w4_matvec(x, qw, qs, y, 32)
    assert bool((y[0] == 64).all()) and bool((y[2] == 64).all()) and bool(torch.isnan(y[1]).all())


# ------------------------------------------------------------------------------ all of them
def _each(run):
    """Calls run(name, call) with a call of each layer that writes (y, state or y)."""
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    c, n, length = 264, 16, 700
    x, w, dt, b, cc = r(2, length, c), r(c, 4), r(2, length, c), r(2, length, n), r(2, length, n)
    a = -torch.rand((c, n), generator=g, device="cuda")
    qw = torch.randint(0, 256, (999, 512), generator=g, device="cuda", dtype=torch.uint8)
    qs, xt = r(999, 8), r(3, 1024)

    def conv():
        y, st = torch.full_like(x, 9.0), torch.zeros((2, 3, c), dtype=x.dtype, device="cuda")
        return lambda: fcm.causal_conv(x, w, y, state_in=st, state_out=st), y, st

    def scan():
        y, st = torch.full_like(x, 9.0), torch.zeros((2, c, n), device="cuda")
        return lambda: fcm.selective_scan(x, dt, a, b, cc, y, state_in=st, state_out=st), y, st

    def w4():
        y = torch.full((3, 999), 9.0, dtype=x.dtype, device="cuda")
        return lambda: fcm.w4_matvec(xt, qw, qs, y, 128), y, y
    for make in (conv, scan, w4):
        run(make)


def test_the_same_bits_every_time():
    def run(make):
        first = None
        for _ in range(4):
            call, y, st = make()
            call()
            got = y.clone(), st.clone()
            if first is not None:
                assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])
            first = got
    _each(run)


def test_on_another_stream_and_in_a_graph():
    """The call runs on the current stream, or the one given, and can be captured."""
    def run(make):
        call, y, st = make()
        call()
        torch.cuda.synchronize()
        want = y.clone()
        call, y, st = make()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            y.fill_(9.0)            # late on this stream: a call on another one would be overwritten
            call()
        side.synchronize()
        assert torch.equal(y, want)
        call, y, st = make()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        st.zero_()
        y.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    _each(run)


def test_each_call_sees_the_one_before():
    """Launches may overlap; what a call reads from the one before must be finished."""
    c, n, steps = 520, 16, 50
    g = np.random.default_rng(11)
    x, dt, a, bm, cm, sk, zz, bi = scan_inputs(g, steps, c, n, 1, "f32")
    w, wh = dev(g.standard_normal((c, 4)) * 0.3, "f32")
    conv, scan = torch.zeros((1, 3, c), device="cuda"), torch.zeros((1, c, n), device="cuda")
    mid, y = torch.empty((steps, c), device="cuda"), torch.empty((steps, c), device="cuda")
    torch.cuda.synchronize()
    for t in range(steps):
        p = slice(t, t + 1)
        fcm.causal_conv(x[0][None, p], w, mid[None, p], act="relu", state_in=conv, state_out=conv)
        fcm.selective_scan(mid[None, p], dt[0][None, p], a[0], bm[0][None, p], cm[0][None, p],
                           y[None, p], skip=sk[0], dt_bias=bi[0], state_in=scan, state_out=scan)
    want, e, _ = ref.causal_conv(x[1], wh, None, None, "relu", [(0, steps)], None, None, 1, "f32")
    within(mid, want, e, "convolution")
    want, e, _, _ = ref.selective_scan(mid.double().cpu().numpy(), dt[1], a[1], bm[1], cm[1], sk[1],
                                       None, bi[1], True, [(0, steps)], None, None, 1, "f32")
    within(y, want, e, "scan")


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Rows more than 2^32 elements from the first one."""
    ld, rows, c, n = 1 << 22, 1200, 24, 16
    wide = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    x, y1, y2 = (wide[:, i * 64:i * 64 + c] for i in range(3))
    b = wide[:, 256:256 + n]
    small = torch.randn((rows, c), device="cuda").bfloat16()
    bs = torch.randn((rows, n), device="cuda").bfloat16()
    x.copy_(small)
    b.copy_(bs)
    w = torch.randn((c, 4), device="cuda").bfloat16()
    a = -torch.rand((c, n), device="cuda")
    want = torch.empty_like(small)
    fcm.causal_conv(x[None], w, y1[None])
    fcm.causal_conv(small[None], w, want[None])
    assert torch.equal(y1, want)
    fcm.selective_scan(x[None], x[None], a, b[None], b[None], y2[None])
    fcm.selective_scan(small[None], small[None], a, bs[None], bs[None], want[None])
    assert torch.equal(y2, want)
