"""silu and its gate over all of its range, in 32 bits.  Where the logistic factor is below the least normal
float, 2^-126, the result is 0, which is off by less than 2^-126 times v; everywhere else it is within the
roundings' bound."""
import numpy as np
import pytest

import pointwise_conv_cnn_gb300 as fcm
import seq_reference as ref
import seq_wide as wide

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def lost(v):
    """What is lost of v times a factor that is below 2^-126 (or is 400 units of rounding above it)."""
    return torch.where(v.double() < -87.33, v.double().abs() * torch.minimum(torch.sigmoid(v.double()), torch.tensor(
        2.0 ** -126 * (1 + 400 * ref.U), dtype=torch.float64, device=v.device)), 0.0)


def values():
    v = np.concatenate([np.linspace(-110.0, 110.0, 4401), np.linspace(-92.0, -86.0, 601),
                        np.geomspace(1e-37, 1.0, 300), -np.geomspace(1e-37, 1.0, 300), [0.0, 1e30, 3e38]])
    v = np.concatenate([v, np.zeros(-len(v) % 8)])   # whole rows of 8 channels
    return torch.from_numpy(v).float().cuda()


@pytest.mark.parametrize("c", [8, 1])   # 16 bytes, and one channel, a thread
def test_activation(c):
    v = values().view(1, -1, c)
    y = torch.empty_like(v)
    fcm.causal_conv(v, torch.ones((c, 1), device="cuda"), y, act="silu")
    want, e = wide.act(v.double(), torch.zeros_like(v, dtype=torch.float64), "silu")
    wide.within(y, want, wide.stored(want, e, "f32") + lost(v), "silu")


@pytest.mark.parametrize("length", [1, 0])   # single tokens, one prompt (0: all rows)
def test_gate(length):
    """One state that takes x as it is, y = x * silu(z)."""
    z = values().view(-1, 8)
    z = z.unsqueeze(1) if length else z.unsqueeze(0)
    one = torch.ones((*z.shape[:2], 1), device="cuda")
    x, y = torch.ones_like(z), torch.empty_like(z)
    fcm.selective_scan(x, torch.ones_like(z), torch.full((8, 1), -200.0, device="cuda"), one, one, y, z=z, softplus=False)
    want, e = wide.act(z.double(), torch.zeros_like(z, dtype=torch.float64), "silu")
    wide.within(y, want, wide.stored(want, e + 8 * ref.U * want.abs(), "f32") + lost(z), "gate")
