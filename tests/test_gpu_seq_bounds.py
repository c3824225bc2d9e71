"""max_len is a bound of the packed sequences' lengths: one that is not the longest length, and be it the
greatest int, changes nothing, and sequences may be as long as an int counts."""
import pytest

import pointwise_conv_cnn_gb300 as fcm
from launches import launch_of

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]
GREATEST = 2 ** 31 - 1


def conv(lengths, c, dtype, max_len, k=4):
    g = torch.Generator("cuda").manual_seed(c)
    tokens = sum(lengths)
    x, w = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((tokens, c), (c, k)))
    y = torch.full_like(x, 7.0)
    out = torch.full((len(lengths), k - 1, c), 7.0, dtype=dtype, device="cuda")
    start = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    return lambda stream=None: fcm.causal_conv(x, w, y, seq_start=start, max_len=max_len, state_out=out, stream=stream), y, out


def scan(lengths, c, dtype, max_len, n=16):
    g = torch.Generator("cuda").manual_seed(c)
    tokens = sum(lengths)
    x, dt, b, cc = (torch.randn((tokens, s), generator=g, device="cuda").to(dtype) for s in (c, c, n, n))
    a = -torch.rand((c, n), generator=g, device="cuda")
    y, out = torch.full_like(x, 7.0), torch.full((len(lengths), c, n), 7.0, device="cuda")
    start = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    return lambda stream=None: fcm.selective_scan(x, dt, a, b, cc, y, seq_start=start, max_len=max_len, state_out=out,
                                                  stream=stream), y, out


@pytest.mark.parametrize("layer", [conv, scan], ids=["conv", "scan"])
@pytest.mark.parametrize("lengths,c", [([40, 60], 4096), ([3, 0, 200, 1], 100), ([1, 1, 1], 33), ([0, 0], 64), ([700], 40)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_loose_bounds(layer, lengths, c, dtype):
    """None (the binding's: all tokens), the tokens, and past them, up to what an int holds."""
    exact = layer(lengths, c, dtype, max(lengths))
    exact[0]()
    grids = set()
    for max_len in (None, sum(lengths), sum(lengths) + 5, 2 ** 30, GREATEST - 30, GREATEST):
        call, y, out = layer(lengths, c, dtype, max_len)
        grids.add(launch_of(call).grid)
        call()
        torch.cuda.synchronize()
        if layer is conv:
            assert torch.equal(y, exact[1]) and torch.equal(out, exact[2])
        else:   # another bound may choose another shape, whose sums run in another order
            tol = dict(rtol=2.0 ** -7 if dtype == torch.bfloat16 else 1e-4, atol=1e-3)
            torch.testing.assert_close(y, exact[1], **tol)
            torch.testing.assert_close(out, exact[2], **tol)
    assert len(grids) == 1, grids


@pytest.mark.slow
@pytest.mark.parametrize("packed", [False, True])
def test_conv_of_the_longest_sequence(packed):
    """2^31 - 1 rows of one channel: the last tile ends where an int does."""
    rows, piece = GREATEST, 1 << 24
    x = torch.empty((rows, 1), dtype=torch.bfloat16, device="cuda")
    for at in range(0, rows, piece):
        x[at:at + piece].normal_(generator=torch.Generator("cuda").manual_seed(at // piece))
    w = torch.randn((1, 4), device="cuda").bfloat16()
    y = torch.full_like(x, float("nan"))
    out = torch.empty((1, 3, 1), dtype=torch.bfloat16, device="cuda")
    if packed:
        fcm.causal_conv(x, w, y, act="none", state_out=out, seq_start=torch.tensor([0, rows], dtype=torch.int32, device="cuda"))
    else:
        fcm.causal_conv(x[None], w, y[None], act="none", state_out=out)
    assert torch.equal(out[0], x[-3:])
    for at in range(0, rows, piece):
        xx = torch.cat((x.new_zeros((3, 1)), x[:piece])) if at == 0 else x[at - 3:at + piece]
        want = sum(w[0, j].double() * xx[j:len(xx) - 3 + j].double() for j in range(4))
        got = y[at:at + piece].double()
        # four products' sum in 32 bits, rounded once
        bound = 2.0 ** -8 * (want.abs() + 1e-5) + 1e-5
        assert bool(((got - want).abs() <= bound).all()), at


def test_binding_takes_the_greatest_bound_and_no_more():
    call, _, _ = conv([5, 2], 16, torch.float32, GREATEST + 1)
    with pytest.raises(fcm.FcmError) as e:
        call()
    assert e.value.status == 1
