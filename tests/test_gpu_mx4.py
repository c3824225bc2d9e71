"""Microscaled 4-bit floating point on the GPU: codes and values equal the definition's, products within the
bound of 32-bit sums (tests/block_reference.py)."""
import numpy as np
import pytest

import block_reference as ref
import pointwise_conv_cnn_gb300 as fcm
from helpers import torch_dtype
from test_gpu_seq_layers import beside, dev, within

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def bytes_like(shape):
    """uint8 tensor between guards."""
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")

    def check():
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + n:] == 0xA5).all())
    return buf[256:256 + n].view(shape), check


def quantised(x):
    q, cq = bytes_like((x.shape[0], x.shape[1] // 2))
    s, cs = bytes_like((x.shape[0], x.shape[1] // 32))
    fcm.mx4_quantize(x, q, s)
    torch.cuda.synchronize()
    cq(), cs()
    return q, s


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 32), (3, 64), (13, 32 * 9), (200, 160), (1, 4096), (65, 32 * 33)])
@pytest.mark.parametrize("left,right", [(0, 0), (8, 0), (3, 2)])
def test_quantise_and_widen(m, k, dtype, left, right):
    g = np.random.default_rng(m + k)
    x = g.standard_normal((m, left + k + right)) * np.exp(2.0 * g.standard_normal((m, 1)))
    x[:, left:left + 32] *= 2.0 ** -6
    xd, xh = dev(x, dtype)
    q, s = quantised(xd[:, left:left + k])
    codes, scale = ref.mx4_quantize(xh[:, left:left + k])
    np.testing.assert_array_equal(s.cpu().numpy(), scale)
    np.testing.assert_array_equal(ref.unpack(q.cpu().numpy()), codes)
    y, unharmed = beside(m, k, dtype, left, right)
    fcm.mx4_dequantize(q, s, y)
    torch.cuda.synchronize()
    unharmed()
    want, _ = dev(ref.mx4_values(codes, scale), dtype)
    assert bool((y == want).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_borders(dtype):
    """Every value halfway between two of the grid, the ones beside it in the storage type, and signs."""
    grid = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0])
    eps = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}[dtype]
    rows = [np.concatenate([[4.0], grid[1:] * f]) for f in (1.0, 1 - eps, 1 + eps)]   # the first sets the power
    x = np.stack([np.concatenate([r, -r]) for r in rows])
    x = np.concatenate([x, x * 2.0 ** -9, x * 2.0 ** 7])
    xd, xh = dev(x, dtype)
    q, s = quantised(xd)
    codes, scale = ref.mx4_quantize(xh)
    np.testing.assert_array_equal(s.cpu().numpy(), scale)
    np.testing.assert_array_equal(ref.unpack(q.cpu().numpy()), codes)


def test_zeros_small_large_and_what_is_no_number():
    tiny, big = 2.0 ** -140, 3.0e38
    x = np.zeros((8, 64))
    x[1, :32], x[2, 5], x[3, :32], x[4, 40] = tiny, 2.0 ** -126, big, 1.0
    x[5, 7], x[6, 33], x[7, :2] = np.inf, np.nan, [-np.inf, 1.0]
    xd, xh = dev(x, "f32")
    q, s = quantised(xd)
    codes, scale = ref.mx4_quantize(xh)
    np.testing.assert_array_equal(s.cpu().numpy(), scale)
    np.testing.assert_array_equal(ref.unpack(q.cpu().numpy()), codes)
    assert scale[5, 0] == 255 and scale[6, 1] == 255 and scale[7, 0] == 255 and scale[0, 0] == 0
    y = torch.empty_like(xd)
    fcm.mx4_dequantize(q, s, y)
    np.testing.assert_array_equal(y.double().cpu().numpy(), ref.mx4_values(codes, scale))


def test_every_code_and_power_widens():
    codes = np.tile(np.arange(16), (256, 2))
    scale = np.arange(256)[:, None]
    q = torch.from_numpy(ref.pack(codes)).cuda()
    s = torch.from_numpy(scale.astype(np.uint8)).cuda()
    for dtype in ("f32", "f16", "bf16"):
        y = torch.empty((256, 32), dtype=torch_dtype(dtype), device="cuda")
        fcm.mx4_dequantize(q, s, y)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(ref.mx4_values(codes, scale)).float().to(torch_dtype(dtype)).double().numpy()
        np.testing.assert_array_equal(y.double().cpu().numpy(), want)


def rows_of(g, m, k, spread=1.0):
    """Random codes, powers near 1."""
    codes = g.integers(0, 16, (m, k))
    scale = np.clip(127 + np.rint(spread * g.standard_normal((m, k // 32))), 0, 254).astype(np.int64)
    return torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scale.astype(np.uint8)).cuda(), ref.mx4_values(codes, scale)


def run_matmul(m, out, k, dtype="bf16", act="none", scale=False, bias=False, left=0, right=0, seed=0, stream=None):
    g = np.random.default_rng(seed)
    xq, xs, x = rows_of(g, m, k)
    wq, ws, w = rows_of(g, out, k)
    sd, sh = dev(g.uniform(0.5, 1.5, out) / np.sqrt(k), "f32") if scale else (None, None)
    bd, bh = dev(g.standard_normal(out), "f32") if bias else (None, None)
    y, unharmed = beside(m, out, dtype, left, right)
    fcm.mx4_matmul(xq, xs, wq, ws, y, scale=sd, bias=bd, act=act, stream=stream)
    torch.cuda.synchronize()
    unharmed()
    want, e = ref.mx4_matmul(x, w, sh, bh, act, dtype)
    within(y, want, e, "y")
    return y


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 127, 128, 130, 257, 300])
@pytest.mark.parametrize("out,k", [(1, 32), (100, 64), (128, 256), (5, 4096), (129, 32 * 9), (515, 1024), (1000, 32 * 17)])
def test_matmul(m, out, k):
    run_matmul(m, out, k, seed=m + out, scale=True, bias=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "relu6", "silu"])
@pytest.mark.parametrize("m", [3, 150])
def test_matmul_options(dtype, act, m):
    run_matmul(m, 200, 288, dtype, act, scale=True, bias=act != "none")


@pytest.mark.parametrize("left,right", [(8, 8), (1, 0), (3, 2), (64, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [5, 140])
def test_matmul_column_blocks(left, right, dtype, m):
    run_matmul(m, 260, 96, dtype, left=left, right=right, scale=True)


@pytest.mark.parametrize("m,out,k", [(16, 4096, 8192), (1, 2048, 4096), (700, 1500, 2048), (1500, 700, 32 * 65), (40, 3000, 32 * 130)])
def test_matmul_large(m, out, k):
    run_matmul(m, out, k, seed=k, scale=True)


@pytest.mark.parametrize("m", [4, 200])
def test_matmul_exact(m):
    """Whole numbers whose sums 32 bits hold: every product is the same in any order."""
    g = np.random.default_rng(3)
    x, w = (g.integers(-1, 2, (r, 512)).astype(np.float64) * 4.0 for r in (m, 300))
    (xq, xs), (wq, ws) = quantised(dev(x, "f32")[0]), quantised(dev(w, "f32")[0])
    y = torch.empty((m, 300), device="cuda")
    fcm.mx4_matmul(xq, xs, wq, ws, y)
    np.testing.assert_array_equal(y.double().cpu().numpy(), x @ w.T)


@pytest.mark.parametrize("m", [4, 200])
def test_matmul_nan_stays_in_its_row(m):
    g = np.random.default_rng(4)
    xq, xs, _ = rows_of(g, m, 256)
    wq, ws, _ = rows_of(g, 140, 256)
    xs[2, 3] = 255
    ws[7, 0] = 255
    y = torch.empty((m, 140), device="cuda")
    fcm.mx4_matmul(xq, xs, wq, ws, y)
    nan = torch.zeros((m, 140), dtype=torch.bool, device="cuda")
    nan[2], nan[:, 7] = True, True
    assert bool((torch.isnan(y) == nan).all())


@pytest.mark.parametrize("power", [-60, 50])
def test_matmul_powers_far_from_one(power):
    """Powers whose product is the result's: nothing is lost on the way."""
    g = np.random.default_rng(5)
    for m in (4, 200):
        xq, xs, x = rows_of(g, m, 256)
        wq, ws, w = rows_of(g, 140, 256)
        y = torch.empty((m, 140), device="cuda")
        xs, ws = (xs.int() + power).to(torch.uint8), (ws.int() + power).to(torch.uint8)
        fcm.mx4_matmul(xq, xs, wq, ws, y)
        want, e = ref.mx4_matmul(x * 2.0 ** power, w * 2.0 ** power, None, None, "none", "f32")
        within(y, want, e, "y")


@pytest.mark.parametrize("m", [5, 300])
def test_matmul_repeats_bit_for_bit_on_streams_and_in_a_graph(m):
    g = np.random.default_rng(7)
    xq, xs, _ = rows_of(g, m, 1024)
    wq, ws, _ = rows_of(g, 600, 1024)

    def call(stream=None):
        y = torch.empty((m, 600), device="cuda", dtype=torch.bfloat16)
        fcm.mx4_matmul(xq, xs, wq, ws, y, act="silu", stream=stream)
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


def test_quantise_in_a_graph_and_on_a_stream():
    x = torch.randn(70, 320, device="cuda", dtype=torch.bfloat16)
    q, s = quantised(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    fcm.mx4_quantize(x, q2, s2, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    q3, s3, y3 = torch.zeros_like(q), torch.zeros_like(s), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        fcm.mx4_quantize(x, q3, s3)
        fcm.mx4_dequantize(q3, s3, y3)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in ((q2, s2), (q3, s3)):
        assert bool((a == q).all()) and bool((b == s).all())
    y = torch.empty_like(x)
    fcm.mx4_dequantize(q, s, y)
    assert bool((y == y3).all())
