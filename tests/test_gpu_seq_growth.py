"""Scans whose sequences are split over parts, with states that grow, that are infinite, or that wait
at zero or at next to nothing for a part's rows: what a part makes of the state before it must not
depend on its factor alone being a float."""
import pytest

import pointwise_conv_cnn_gb300 as fcm
import seq_wide as wide
from helpers import torch_dtype
from launches import launch_of

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]

LENGTH, C, PARTS = 1000, 40, 8
PART = 128   # rows of a part: a tile's 16 or 32 rows divide it
SHAPES = [(16, "f32"), (16, "bf16"), (12, "f32"), (5, "f16"), (64, "f32"), (128, "f32")]


def run(n, dtype, dt, a, x, old):
    """One sequence with B and C of ones' size; returns y, the state after, and the inputs in 64 bits."""
    g = torch.Generator("cuda").manual_seed(n)
    store = torch_dtype(dtype)
    x, dt = x.to(store), dt.to(store)
    bm, cm = (torch.rand((1, LENGTH, n), generator=g, device="cuda").add(0.5).to(store) for _ in range(2))
    y, out = torch.empty_like(x), torch.empty((1, C, n), device="cuda")

    def call(stream=None):
        fcm.selective_scan(x, dt, a, bm, cm, y, softplus=False, state_in=old, state_out=out, stream=stream)
    assert launch_of(call).cluster == PARTS, "the sequence is not split"
    call()
    torch.cuda.synchronize()
    d = [v.double() for v in (x[0], dt[0], a, bm[0][:, None], cm[0][:, None])]
    return y[0], out, d


def check(n, dtype, dt, a, x, old=None):
    y, out, d = run(n, dtype, dt, a, x, old)
    want, e, h, e_h = wide.scan(*d, None, None, None, False, [LENGTH], None if old is None else old.double(),
                                dtype, part_rows=PART)
    assert bool(torch.isfinite(want).all()) and bool(torch.isfinite(h).all())
    wide.within(y, want, e, "y")
    wide.within(out, h, e_h, "state")


def steps(big_rows, big, small=2.0 ** -7):
    dt = torch.full((1, LENGTH, C), small, device="cuda")
    dt[:, big_rows] = big
    return dt


@pytest.mark.parametrize("n,dtype", SHAPES)
def test_a_state_of_zero_stays_zero_whatever_its_factor(n, dtype):
    """Nothing comes in for most of the rows, while the factors of whole parts pass what a float holds."""
    x = torch.zeros((1, LENGTH, C), device="cuda")
    x[:, 900:] = torch.randn((100, C), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    check(n, dtype, steps(slice(0, 850), 1.0), torch.ones((C, n), device="cuda"), x)


@pytest.mark.parametrize("n,dtype", SHAPES)
def test_a_small_state_grows_to_what_it_should(n, dtype):
    """1e-30 times e^100 within one part, whose factor by itself is past 32 bits."""
    x = torch.zeros((1, LENGTH, C), device="cuda")
    old = torch.full((1, C, n), 1e-30, device="cuda")
    dt = steps(slice(200, 240), 2.5, 2.0 ** -13)
    if dtype == "f16":   # y stays within f16: 1e-37 times e^90
        old.fill_(1e-37)
        dt = steps(slice(200, 240), 2.25, 2.0 ** -13)
    check(n, dtype, dt, torch.ones((C, n), device="cuda"), x, old)


@pytest.mark.parametrize("n,dtype", SHAPES)
def test_a_large_state_falls_to_what_it_should(n, dtype):
    """1e30 times e^-100 within one part."""
    x = torch.zeros((1, LENGTH, C), device="cuda")
    old = torch.full((1, C, n), 1e30, device="cuda")
    if dtype == "f16":
        old.fill_(1e3)
    check(n, dtype, steps(slice(200, 240), 2.5, 2.0 ** -13), -torch.ones((C, n), device="cuda"), x, old)


@pytest.mark.parametrize("n,dtype", SHAPES)
def test_steps_of_either_sign(n, dtype):
    """Growth and decay by turns, over all parts."""
    g = torch.Generator("cuda").manual_seed(7)
    x = torch.randn((1, LENGTH, C), generator=g, device="cuda")
    dt = 0.0625 * torch.randn((1, LENGTH, C), generator=g, device="cuda")
    check(n, dtype, dt, 0.2 + 0.5 * torch.rand((C, n), generator=g, device="cuda"), x,
          torch.randn((1, C, n), generator=g, device="cuda"))


@pytest.mark.parametrize("n,dtype", SHAPES)
def test_an_infinite_state_stays_infinite(n, dtype):
    """Each row's factor is e^-1; a part's is nothing.  The other channels stay as they are."""
    x = torch.ones((1, LENGTH, C), device="cuda")
    old = torch.ones((1, C, n), device="cuda")
    old[0, 3], old[0, 7] = float("inf"), float("-inf")
    y, out, _ = run(n, dtype, steps(slice(0, LENGTH), 1.0), -torch.ones((C, n), device="cuda"), x, old)
    inf = float("inf")
    assert bool((out[0, 3] == inf).all()) and bool((y[:, 3] == inf).all())
    assert bool((out[0, 7] == -inf).all()) and bool((y[:, 7] == -inf).all())
    rest = torch.ones(C, dtype=torch.bool, device="cuda")
    rest[3] = rest[7] = False
    assert bool(torch.isfinite(out[0, rest]).all()) and bool(torch.isfinite(y[:, rest]).all())


@pytest.mark.parametrize("n,dtype", SHAPES)
def test_nan_goes_on_from_where_it_is(n, dtype):
    """A step that is no number makes its channel's states none from its row on, and no other's."""
    dt = steps(slice(0, 0), 0.0)
    dt[0, 300, 5] = float("nan")
    y, out, _ = run(n, dtype, dt, -torch.ones((C, n), device="cuda"), torch.ones((1, LENGTH, C), device="cuda"), None)
    assert bool(torch.isfinite(y[:300]).all()) and bool(torch.isnan(y[300:, 5]).all()) and bool(torch.isnan(out[0, 5]).all())
    y[:, 5], out[:, 5] = 0, 0
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(out).all())
