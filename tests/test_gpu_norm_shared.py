"""Group normalisation of samples that clusters share: two kernels, the first of which leaves the groups' sums in the
outputs.  Every variant that the rule chooses, against 64 bits (tests/block_reference.py)."""
import numpy as np
import pytest

import block_reference as ref
import pointwise_conv_cnn_gb300 as fcm
from helpers import torch_dtype
from launches import captured
from test_gpu_seq_layers import dev, within

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def run(n, pixels, c, groups, dtype, vector, act="none", affine=True, gate=False, rms=False, left=0, right=0, shift=0, mean=1.0,
        samples=None):
    """x and z are column blocks [left, left + c) of wider rows, y rows of c, `shift` elements behind an aligned
    address, between guards; `samples` are compared (all), `vector` channels at once are expected."""
    g = np.random.default_rng(c + pixels)
    wide = left + c + right

    def rows(values):
        d, h = dev(values.reshape(n, pixels, wide), dtype)
        return d[..., left:left + c], h[..., left:left + c]
    x, xh = rows(g.standard_normal((n * pixels, wide)) * g.uniform(0.5, 2.0, wide) + mean * g.standard_normal(wide))
    z, zh = rows(g.standard_normal((n * pixels, wide))) if gate else (None, None)
    s, sh = dev(g.uniform(0.5, 1.5, c), "f32") if affine else (None, None)
    b, bh = dev(g.standard_normal(c), "f32") if affine else (None, None)
    size = n * pixels * c
    buf = torch.full((size + 256,), 7.0, dtype=torch_dtype(dtype), device="cuda")
    y = buf[64 + shift:64 + shift + size].view(n, pixels, c)

    def call(stream=None):
        fcm.group_norm(x, y, groups, scale=s, bias=b, act=act, z=z, rms=rms, stream=stream)
    kernels = captured(call)
    assert [k.numbers[:2] for k in kernels] == [(vector, 0 if z is None else 1)] * 2, kernels
    assert "norm_maps" in kernels[0].name and "norm_apply" in kernels[1].name
    call()
    first = y.clone()
    call()   # over the first's outputs
    torch.cuda.synchronize()
    assert bool((y == first).all())
    assert bool((buf[:64 + shift] == 7.0).all()) and bool((buf[64 + shift + size:] == 7.0).all())
    pick = list(range(n)) if samples is None else samples
    want, e = ref.group_norm(xh[pick], groups, sh, bh, float(np.float32(1e-5)), act, None if z is None else zh[pick], rms, dtype)
    within(y[pick], want, e, "y")


@pytest.mark.parametrize("gate,rms,act", [(False, False, "silu"), (True, False, "none"), (False, True, "relu"), (True, True, "relu6")])
@pytest.mark.parametrize("dtype,vector", [("bf16", 8), ("f32", 4)])
def test_gate_and_mean(dtype, vector, gate, rms, act):
    run(2, 200 * 200, 256, 32, dtype, vector, act=act, gate=gate, rms=rms)


@pytest.mark.parametrize("gate,rms", [(False, False), (True, True)])
@pytest.mark.parametrize("n,pixels,c,groups,dtype,vector", [
    (3, 10000, 599, 1, "bf16", 1),      # odd channels
    (2, 130000, 66, 11, "f16", 2),      # pairs of channels, groups of 6
    (1, 40000, 66, 66, "bf16", 2),      # a channel a group
    (2, 60000, 77, 7, "f32", 1),
    (1, 4096, 2048, 2048, "bf16", 8),   # the most groups: 192 pixels hold their sums
    (1, 4097, 2048, 16, "f16", 8),      # some clusters have no pixel
    (25, 6000, 64, 8, "f32", 4),        # three clusters a sample
    (1, 70001, 120, 5, "bf16", 8)])
def test_shapes(n, pixels, c, groups, dtype, vector, gate, rms):
    run(n, pixels, c, groups, dtype, vector, gate=gate, rms=rms, act="silu")


def test_one_cluster_a_sample():
    run(80, 6000, 64, 8, "f32", 4, gate=True, samples=[0, 1, 41, 79])


@pytest.mark.parametrize("dtype,left,right,vector", [("bf16", 8, 8, 8), ("bf16", 64, 0, 8), ("bf16", 2, 4, 2), ("bf16", 1, 0, 1),
                                                     ("f16", 0, 3, 1), ("f32", 4, 8, 4), ("f32", 1, 2, 1)])
def test_inputs_that_are_column_blocks(dtype, left, right, vector):
    run(2, 36000 if dtype == "f32" else 72000, 128, 16, dtype, vector, left=left, right=right, gate=True, act="silu")


@pytest.mark.parametrize("dtype,shift,vector", [("bf16", 1, 1), ("bf16", 2, 2), ("bf16", 7, 1), ("bf16", 8, 8), ("f32", 1, 1), ("f32", 2, 1),
                                                ("f32", 4, 4)])
def test_outputs_off_16_bytes(dtype, shift, vector):
    """The sums begin at the first 16-byte boundary of each sample's outputs."""
    run(2 if shift < 3 else 1, 70000, 127 if vector == 1 else 128, 1, dtype, vector, shift=shift)


@pytest.mark.parametrize("mean", [100.0, 3000.0])
def test_large_means(mean):
    run(2, 36000, 128, 16, "f32", 4, mean=mean, affine=False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_stays_in_its_sample_and_group(bad):
    x = torch.randn((2, 70000, 128), device="cuda").bfloat16()
    y, fine = torch.empty_like(x), torch.ones((2, 70000, 128), dtype=torch.bool, device="cuda")
    x[1, 69999, 20] = bad
    fine[1, :, 16:32] = False
    assert len(captured(lambda s: fcm.group_norm(x, y, 8, stream=s))) == 2
    fcm.group_norm(x, y, 8)
    assert bool(torch.isfinite(y[fine]).all()) and bool(torch.isnan(y[~fine]).all())
