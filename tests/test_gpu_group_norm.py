"""Group normalisation on the GPU against 64 bits, each element within the bound that the computation's own
roundings give (tests/block_reference.py)."""
import numpy as np
import pytest

import block_reference as ref
import pointwise_conv_cnn_gb300 as fcm
from helpers import guarded_empty, torch_dtype
from test_gpu_seq_layers import dev, within

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def run_norm(n, pixels, c, groups, dtype, act="none", scale=True, bias=True, gate=False, rms=False, eps=1e-5, left=0, right=0,
             seed=0, mean=1.0, in_place=False, x=None, stream=None):
    g = np.random.default_rng(seed)
    wide = left + c + right

    def rows(values):
        d, h = dev(values, dtype)
        return d.view(n, pixels, wide)[..., left:left + c], h.reshape(n, pixels, wide)[..., left:left + c]
    if x is None:
        x = g.standard_normal((n * pixels, wide)) * g.uniform(0.5, 2.0, wide) + mean * g.standard_normal(wide)
    xd, xh = rows(x)
    sd, sh = dev(g.uniform(0.5, 1.5, c), "f32") if scale else (None, None)
    bd, bh = dev(g.standard_normal(c), "f32") if bias else (None, None)
    zd, zh = rows(g.standard_normal((n * pixels, wide))) if gate else (None, None)
    if in_place:
        y, unharmed = xd, lambda: None
    else:
        t, check = guarded_empty((n, pixels, wide), dtype, fill=7.0)
        y = t[..., left:left + c]

        def unharmed():
            check()
            assert bool((t[..., :left] == 7.0).all()) and bool((t[..., left + c:] == 7.0).all())
    fcm.group_norm(xd, y, groups, scale=sd, bias=bd, eps=eps, act=act, z=zd, rms=rms, stream=stream)
    torch.cuda.synchronize()
    unharmed()
    want, e = ref.group_norm(xh, groups, sh, bh, float(np.float32(eps)), act, zh, rms, dtype)
    within(y, want, e, "y")
    return y


SHAPES = [(1, 1, 8, 1), (2, 9, 16, 4), (3, 49, 96, 32), (1, 196, 32, 8), (2, 1000, 128, 32), (1, 5000, 64, 1), (2, 33, 30, 3),
          (1, 77, 1, 1), (4, 10, 512, 512), (1, 300, 1021, 1), (1, 20, 6000, 2), (17, 5, 40, 10)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,pixels,c,groups", SHAPES)
@pytest.mark.parametrize("rms", [False, True])
def test_maps(n, pixels, c, groups, dtype, rms):
    run_norm(n, pixels, c, groups, dtype, rms=rms, seed=c)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,groups,each", [(1, 1, 128), (5, 32, 128), (37, 4, 64), (3, 7, 96), (9, 3, 100), (2, 5, 33), (4, 2, 256),
                                           (6, 1, 1000), (3, 2, 2048), (5, 3, 250), (8, 16, 8), (3, 40, 1), (2, 1, 5000), (300, 2, 72)])
@pytest.mark.parametrize("gate,rms", [(False, False), (True, True)])
def test_rows(n, groups, each, dtype, gate, rms):
    run_norm(n, 1, groups * each, groups, dtype, gate=gate, rms=rms, seed=each)


@pytest.mark.parametrize("act", ["none", "relu", "relu6", "silu"])
@pytest.mark.parametrize("scale,bias,gate", [(False, False, False), (True, False, True), (False, True, True)])
@pytest.mark.parametrize("pixels", [1, 50])
def test_options(act, scale, bias, gate, pixels):
    run_norm(2, pixels, 48, 6, "f16", act=act, scale=scale, bias=bias, gate=gate)


@pytest.mark.parametrize("left,right", [(8, 8), (1, 0), (0, 1), (4, 12), (64, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pixels", [1, 60])
def test_column_blocks(left, right, dtype, pixels):
    run_norm(2, pixels, 64, 8, dtype, left=left, right=right, gate=True)


@pytest.mark.parametrize("pixels", [1, 60, 40000])
def test_in_place(pixels):
    run_norm(2, pixels, 64, 8, "bf16", in_place=True, act="silu")


@pytest.mark.parametrize("n,pixels,c,groups", [(1, 200 * 200, 128, 32), (2, 16384, 64, 1), (40, 3136, 128, 32), (1, 65537, 24, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_maps(n, pixels, c, groups, dtype):
    """Samples that a cluster shares, kept whole and in part."""
    run_norm(n, pixels, c, groups, dtype, act="silu", gate=pixels < 20000)


@pytest.mark.parametrize("mean", [100.0, 3000.0])
@pytest.mark.parametrize("pixels", [1, 900])
def test_large_means(mean, pixels):
    run_norm(2, pixels, 64, 2, "f32", mean=mean)
    x = np.random.default_rng(9).standard_normal((2 * pixels, 64)) + mean
    run_norm(2, pixels, 64, 2, "f32", x=x)


def test_one_value_far_from_the_others():
    x = np.random.default_rng(10).standard_normal((700, 32))
    x[0, 0] = 1e4
    run_norm(1, 700, 32, 4, "f32", x=x)


@pytest.mark.parametrize("pixels", [1, 30])
def test_equal_values_and_no_eps(pixels):
    run_norm(1, pixels, 32, 4, "bf16", x=np.full((pixels, 32), 3.0))
    run_norm(1, pixels, 32, 4, "bf16", eps=0.0)


@pytest.mark.parametrize("pixels", [1, 40])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_nan_stays_in_its_sample_and_group(pixels, bad):
    x = np.random.default_rng(11).standard_normal((3, pixels, 64))
    x[1, pixels // 2, 20] = bad
    xd, _ = dev(x, "f16")
    y = torch.empty_like(xd)
    fcm.group_norm(xd, y, 8)
    fine = torch.ones((3, pixels, 64), dtype=torch.bool)
    fine[1, :, 16:24] = False
    assert bool(torch.isfinite(y.cpu()[fine]).all()) and bool(torch.isnan(y[1, :, 16:24]).all())


def test_shapes_of_any_number_of_dimensions():
    x = torch.randn(2, 5, 7, 16, device="cuda")
    want = torch.empty(2, 35, 16, device="cuda")
    fcm.group_norm(x.view(2, 35, 16), want, 4)
    for shape in [(2, 5, 7, 16), (2, 5, 1, 7, 16), (2, 35, 1, 16)]:
        y = torch.empty(shape, device="cuda")
        fcm.group_norm(x.view(shape), y, 4)
        assert bool((y.view(2, 35, 16) == want).all())
    rows = torch.empty(70, 16, device="cuda")
    fcm.group_norm(x.view(70, 16), rows, 4)
    one = torch.empty(70, 1, 1, 16, device="cuda")
    fcm.group_norm(x.view(70, 1, 1, 16), one, 4)
    assert bool((rows == one.view(70, 16)).all()) and not bool((rows == want.view(70, 16)).all())


@pytest.mark.parametrize("shape", [(300, 256), (4, 3000, 64)])
def test_repeats_bit_for_bit_on_streams_and_in_a_graph(shape):
    x = torch.randn(shape, device="cuda", dtype=torch_dtype("bf16"))

    def call(stream=None):
        y = torch.empty_like(x)
        fcm.group_norm(x, y, 8, act="silu", stream=stream)
        return y
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [call(side), call(side)]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(call())
    got[-1].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((y == want).all()) for y in got)
