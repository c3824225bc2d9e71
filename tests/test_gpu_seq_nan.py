"""A value that is no number stays none through every activation of the layers over sequences, in its
own outputs only; infinities are cut where the activation cuts them."""
import pytest

import pointwise_conv_cnn_gb300 as fcm
from helpers import torch_dtype

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]
ACTS = {"none": lambda v: v, "relu": torch.relu, "relu6": lambda v: v.clamp(0.0, 6.0), "silu": lambda v: v * torch.sigmoid(v)}


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c", [64, 34, 33])   # 16 bytes, two channels and one channel a thread
def test_conv(c, dtype, act):
    x = torch.ones((1, 20, c), dtype=torch_dtype(dtype), device="cuda")
    x[0, 4, 3], x[0, 5, 7], x[0, 6, 9] = float("nan"), float("inf"), float("-inf")
    w = torch.full((c, 2), 0.5, dtype=x.dtype, device="cuda")
    y = torch.empty_like(x)
    fcm.causal_conv(x, w, y, act=act)
    v = 0.5 * x.double()
    v[:, 1:] += 0.5 * x.double()[:, :-1]
    want = ACTS[act](v)
    assert bool(torch.isnan(want[0, 4:6, 3]).all())
    torch.testing.assert_close(y.double(), want, rtol=2.0 ** -7, atol=0, equal_nan=True)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [3, 12])
def test_w4(m, dtype, act):
    x = torch.ones((m, 64), dtype=torch_dtype(dtype), device="cuda")
    x[1, 5], x[2, 6] = float("nan"), float("inf")
    qw = torch.full((20, 32), 0x99, dtype=torch.uint8, device="cuda")   # weights of 1
    qw[10:] = 0x77                                                      # and of -1
    qs = torch.full((20, 2), 0.25, dtype=x.dtype, device="cuda")
    y = torch.empty((m, 20), dtype=x.dtype, device="cuda")
    fcm.w4_matvec(x, qw, qs, y, 32, act=act)
    sign = torch.ones(20, dtype=torch.float64, device="cuda")
    sign[10:] = -1.0
    want = ACTS[act](0.25 * x.double().sum(1)[:, None] * sign)
    assert bool(torch.isnan(want[1]).all())
    torch.testing.assert_close(y.double(), want, rtol=2.0 ** -7, atol=2.0 ** -24, equal_nan=True)
