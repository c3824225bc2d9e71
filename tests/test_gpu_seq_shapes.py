"""The convolution's and the scan's kernels in every shape that the rules choose between, at sizes that
reach them: each case says which one it means and looks whether that is launched, then compares every element
with 64 bits (tests/seq_wide.py)."""
import pytest

import pointwise_conv_cnn_gb300 as fcm
import seq_wide as wide
from helpers import guarded_empty, torch_dtype
from launches import launch_of

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]
ITEM = {"f32": 4, "f16": 2, "bf16": 2}


def starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


class Random:
    def __init__(self, seed):
        self.g = torch.Generator("cuda").manual_seed(seed)

    def __call__(self, shape, dtype="f32", std=1.0, left=0):
        """A tensor whose rows start `left` elements into those of a wider one, and its values in 64 bits."""
        t = (torch.randn((*shape[:-1], shape[-1] + left), generator=self.g, device="cuda") * std).to(torch_dtype(dtype))[..., left:]
        return t, t.double()

    def uniform(self, shape, lo, hi):
        t = torch.rand(shape, generator=self.g, device="cuda") * (hi - lo) + lo
        return t, t.double()

    def slots(self, n_seq, slots):
        return torch.randperm(slots, generator=self.g, device="cuda")[:n_seq].to(torch.int32)


# ------------------------------------------------------------------------------ convolution
# lengths, channels, taps, type, channels a thread, rows a thread
CONV = [
    ([2100], 4096, 4, "bf16", 8, 32), ([600, 0, 1500, 7], 4096, 4, "f16", 8, 32), ([1040], 2048, 3, "f32", 4, 16),
    ([1100], 4096, 4, "bf16", 8, 16), ([515], 4096, 4, "bf16", 8, 8), ([300, 0, 100, 113], 4096, 2, "f16", 8, 16),
    ([270], 4096, 8, "bf16", 8, 8), ([2100], 4096, 8, "f16", 8, 32), ([300], 4096, 5, "bf16", 8, 4),
    ([1000, 33], 2046, 4, "bf16", 2, 32), ([300], 1022, 4, "f16", 2, 4), ([700], 1022, 6, "f32", 2, 8), ([517, 1, 0], 1022, 3, "bf16", 2, 16),
    ([1000], 1021, 4, "bf16", 1, 32), ([1031, 0, 40], 333, 4, "f16", 1, 32), ([400], 1021, 7, "f32", 1, 8), ([555], 1021, 2, "bf16", 1, 16),
    ([100, 31], 1021, 4, "f32", 1, 4), ([2100], 4096, 1, "bf16", 8, 32)]


@pytest.mark.parametrize("lengths,c,k,dtype,vec,rows", CONV, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_conv(lengths, c, k, dtype, vec, rows, in_place):
    r, tokens, n_seq, slots = Random(c + k), sum(lengths), len(lengths), len(lengths) + 3
    (x, xd), (w, wd), (b, bd) = r((tokens, c), dtype), r((c, k), dtype, k ** -0.5), r((c,))
    s, sd = r.uniform((c,), 0.5, 1.5)
    old, od = r((slots, k - 1, c), dtype)
    slot = r.slots(n_seq, slots)
    y, guards = guarded_empty((tokens, c), dtype, fill=7.0)
    out, out_guards = guarded_empty((slots, k - 1, c), dtype, fill=3.0)
    if in_place:
        out.copy_(old)

    def call(stream=None):
        fcm.causal_conv(x, w, y, scale=s, bias=b, act="silu", seq_start=starts(lengths) if stream is None else at,
                        max_len=max(lengths), slot=slot, state_in=out if in_place else old, state_out=out, stream=stream)
    at = starts(lengths)
    launch = launch_of(call)
    assert launch.numbers[-2:] == (vec, k), launch
    tiles = {n: -(-(n_seq * (c // vec) * -(-max(lengths) // n)) // 128) for n in (4, 8, 16, 32)}
    assert launch.grid[0] == tiles[rows] and len(set(tiles.values())) == 4, (launch, tiles)
    call()
    torch.cuda.synchronize()
    guards(), out_guards()
    want, e, state = wide.conv(xd, wd, sd, bd, "silu", lengths, od[slot.long()], dtype)
    wide.within(y, want, e, "y")
    assert torch.equal(out[slot.long()].double(), state)
    others = torch.ones(slots, dtype=torch.bool, device="cuda")
    others[slot.long()] = False
    assert bool((out[others] == (old[others] if in_place else 3.0)).all())


# ------------------------------------------------------------------------------ scan
def scan_case(lengths, c, n, dtype, groups, left, max_len, check_launch, seed, z=True, in_place=False, part_rows=0):
    r, tokens, n_seq, slots = Random(seed), sum(lengths), len(lengths), len(lengths) + 2
    (x, xd), (dt, dtd), (gate, zd) = (r((tokens, c), dtype, left=left) for _ in range(3))
    (b, bd), (cc, cd) = ((t.unflatten(1, (groups, n)), d.unflatten(1, (groups, n))) for t, d in (
        r((tokens, groups * n), dtype, left=left) for _ in range(2)))
    a, ad = r.uniform((c, n), -16.0, -0.2)
    (skip, sd), (bias, bid) = r((c,)), r.uniform((c,), -5.0, 0.0)
    old, od = r((slots, c, n))
    slot = r.slots(n_seq, slots)
    lost = None
    if n_seq > 2:   # one sequence without a state
        lost = n_seq // 2
        slot[lost] = -1
    y, guards = guarded_empty((tokens, c), dtype, fill=7.0)
    out, out_guards = guarded_empty((slots, c, n), "f32", fill=3.0)
    if in_place:
        out.copy_(old)
    at = starts(lengths)

    def call(stream=None):
        fcm.selective_scan(x, dt, a, b, cc, y, skip=skip, z=gate if z else None, dt_bias=bias, seq_start=at, max_len=max_len,
                           slot=slot, state_in=out if in_place else old, state_out=out, stream=stream)
    check_launch(launch_of(call))
    call()
    torch.cuda.synchronize()
    guards(), out_guards()
    begin = od[slot.long().clamp_min(0)]
    if lost is not None:
        begin[lost] = 0
    want, e, state, e_state = wide.scan(xd, dtd, ad, bd, cd, sd, zd if z else None, bid, True, lengths, begin, dtype, part_rows)
    wide.within(y, want, e, "y")
    kept = [q for q in range(n_seq) if q != lost]
    rows = slot.long()[kept]
    wide.within(out[rows], state[kept], e_state[kept], "state")
    others = torch.ones(slots, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert bool((out[others] == (old[others] if in_place else 3.0)).all())


# lengths, channels, states, type, groups, elements off 16 bytes, states a lane, lanes a channel, PAD, parts
SCAN = [
    ([100, 100], 2500, 3, "bf16", 1, 0, 4, 1, 2, 1), ([100, 100], 2500, 4, "f32", 2, 0, 4, 1, 0, 1),
    ([300, 290], 2500, 4, "f16", 1, 0, 4, 1, 0, 4), ([500], 40, 4, "bf16", 1, 3, 4, 1, 0, 8),
    ([700], 2500, 8, "bf16", 1, 0, 4, 2, 0, 4), ([300], 40, 7, "f16", 1, 0, 4, 2, 2, 8), ([100], 40, 8, "f32", 2, 0, 4, 2, 0, 1),
    ([100], 40, 16, "bf16", 1, 0, 4, 4, 0, 1), ([1000, 999, 998], 512, 12, "f32", 1, 0, 4, 4, 1, 2),
    ([700, 600, 650], 512, 12, "bf16", 1, 0, 4, 4, 1, 4), ([1000], 40, 12, "f16", 1, 0, 4, 4, 1, 8), ([1000], 40, 12, "bf16", 2, 3, 4, 4, 1, 8),
    ([1000], 45, 9, "f32", 1, 0, 4, 4, 2, 8), ([1000, 0, 333], 40, 16, "bf16", 1, 3, 4, 4, 0, 8),
    ([300] * 4, 200, 16, "f32", 1, 0, 4, 4, 0, 4),
    ([100, 95], 2500, 16, "f16", 1, 0, 8, 2, 0, 1), ([100, 95, 0, 33], 5000, 16, "bf16", 1, 0, 8, 2, 0, 1), ([64] * 2, 8192, 16, "bf16", 2, 0, 8, 2, 0, 1),
    ([300] * 8, 40, 16, "bf16", 1, 0, 8, 2, 0, 8), ([300] * 8, 45, 16, "f32", 1, 1, 8, 2, 0, 8), ([777], 768, 16, "f32", 1, 0, 8, 2, 0, 8),
    ([64] * 8, 4096, 16, "bf16", 1, 0, 16, 1, 0, 1), ([64] * 9 + [1], 4095, 16, "f16", 1, 0, 16, 1, 0, 1),
    ([100] * 8, 2500, 16, "f32", 2, 0, 16, 1, 0, 1),
    ([100], 40, 32, "bf16", 1, 0, 4, 8, 0, 1), ([300], 40, 32, "f32", 1, 0, 4, 8, 0, 8), ([1000], 24, 20, "bf16", 1, 0, 4, 8, 1, 8),
    ([1000], 24, 20, "f16", 1, 3, 4, 8, 1, 8), ([300] * 8, 40, 20, "f32", 1, 0, 4, 8, 1, 4), ([700] * 3, 200, 20, "bf16", 1, 0, 4, 8, 1, 4),
    ([1000] * 3, 200, 20, "f32", 1, 0, 4, 8, 1, 2), ([500], 24, 19, "bf16", 1, 0, 4, 8, 2, 8),
    ([100], 2500, 32, "bf16", 1, 0, 8, 4, 0, 1), ([64, 40, 0, 64], 2500, 32, "f16", 1, 0, 8, 4, 0, 1), ([300] * 3, 200, 32, "bf16", 1, 0, 8, 4, 0, 4),
    ([300] * 2, 200, 32, "f32", 1, 0, 8, 4, 0, 8),
    ([100], 40, 64, "f32", 1, 0, 8, 8, 0, 1), ([300], 40, 64, "bf16", 2, 0, 8, 8, 0, 8), ([700] * 3, 200, 40, "f16", 1, 0, 8, 8, 1, 4),
    ([300], 24, 42, "bf16", 1, 1, 8, 8, 2, 8),
    ([100] * 3, 40, 128, "f32", 1, 0, 8, 16, 0, 1), ([100], 40, 128, "bf16", 1, 0, 8, 16, 0, 8), ([300] * 3, 40, 72, "f32", 1, 0, 8, 16, 1, 4),
    ([200], 12, 100, "f16", 1, 3, 8, 16, 2, 8)]


@pytest.mark.parametrize("lengths,c,n,dtype,groups,left,spt,lpc,pad,parts", SCAN, ids=str)
def test_scan(lengths, c, n, dtype, groups, left, spt, lpc, pad, parts):
    def launched(launch):
        assert launch.numbers[-4:] == (spt, lpc, pad, int(parts > 1)) and launch.cluster == parts, launch
    scan_case(lengths, c, n, dtype, groups, left, max(lengths), launched, c + n, z=c % 4 == 0, in_place=len(lengths) % 2 == 1,
              part_rows=-(-max(lengths) // parts) + 32 if parts > 1 else 0)


# sequences, channels, states, type, states four at a time, lanes a channel
TOKENS = [(193, 5120, 16, "bf16", 1, 4), (301, 1030, 24, "f16", 1, 8), (231, 3000, 5, "f32", 0, 2), (235, 3001, 8, "bf16", 1, 2),
          (181, 2050, 13, "bf16", 0, 4), (99, 2048, 33, "f32", 0, 16), (101, 1000, 64, "f16", 1, 16), (51, 1000, 128, "f32", 1, 32),
          (60, 1111, 127, "bf16", 0, 32)]


@pytest.mark.parametrize("n_seq,c,n,dtype,vec,lpc", TOKENS, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_scan_of_single_tokens(n_seq, c, n, dtype, vec, lpc, in_place):
    """Many sequences, so that a block goes from one pair to the next several times, some without a token."""
    lengths = [0 if q % 7 == 3 else 1 for q in range(n_seq)]

    def launched(launch):
        assert launch.numbers[-2:] == (vec, lpc), launch
        turns = launch.grid[0] / -(-c // (128 // lpc))
        assert turns == int(turns) and -(-n_seq // 2) >= 3 * turns, launch
    scan_case(lengths, c, n, dtype, 1, 0, 1, launched, c + n, in_place=in_place)
