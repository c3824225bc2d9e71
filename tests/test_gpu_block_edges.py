"""The gated delta rule, group normalisation and microscaled 4-bit values where offsets pass 32 bits, calls
meet on streams, and devices and addresses are not the usual ones."""
import numpy as np
import pytest

import block_reference as ref
import pointwise_conv_cnn_gb300 as fcm
from launches import captured
from test_gpu_seq_layers import dev, ints, within

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]
FAR = 1 << 31


def far_rows(rows, cols, distance, dtype=torch.bfloat16):
    """`rows` rows of `cols` elements, `distance` elements apart."""
    buf = torch.empty(((rows - 1) * distance + cols,), dtype=dtype, device="cuda")
    return buf.as_strided((rows, cols), (distance, 1))


@pytest.mark.parametrize("length", [5, 40])
def test_delta_rows_far_apart(length):
    """The last rows lie past 2^31 elements: the same as side by side."""
    g = torch.Generator("cuda").manual_seed(1)
    near = {n: torch.randn((length, c), generator=g, device="cuda").bfloat16() for n, c in
            (("q", 64), ("k", 64), ("v", 64), ("dt", 2), ("b", 2))}
    far = {n: far_rows(length, t.shape[1], FAR // (length - 1) + 8).copy_(t) for n, t in near.items()}
    a, got = -torch.ones(2, device="cuda"), []
    for t in (near, far):
        y = torch.empty((length, 64), dtype=torch.bfloat16, device="cuda") if t is near else \
            far_rows(length, 64, FAR // (length - 1) + 8)
        out = torch.empty((1, 2, 32, 32), device="cuda")
        q, k = (t[n].unflatten(1, (2, 32)) for n in "qk")
        fcm.gated_delta(q, k, t["v"].unflatten(1, (2, 32)), t["dt"], a, t["b"], y.unflatten(1, (2, 32)),
                        seq_start=ints([0, length]), state_out=out)
        got.append((y, out))
    assert bool((got[0][0] == got[1][0]).all()) and bool((got[0][1] == got[1][1]).all())


@pytest.mark.parametrize("length", [1, 40])
def test_delta_states_far_apart(length):
    """Slots past 2^31 elements of the pool."""
    slots = (FAR // (64 * 64)) + 3
    pool = torch.empty((slots, 1, 64, 64), device="cuda")
    pool[[5, slots - 1]] = torch.randn((2, 1, 64, 64), device="cuda")
    old = pool[[5, slots - 1]].clone()
    g = torch.Generator("cuda").manual_seed(2)
    q, k, v = (torch.randn((2, length, 1, 64), generator=g, device="cuda").bfloat16() for _ in range(3))
    dt, b = (torch.randn((2, length, 1), generator=g, device="cuda").bfloat16() for _ in range(2))
    a, y, z, out = -torch.ones(1, device="cuda"), torch.empty_like(v), torch.empty_like(v), torch.empty_like(old)
    fcm.gated_delta(q, k, v, dt, a, b, y, state_in=old, state_out=out)
    fcm.gated_delta(q, k, v, dt, a, b, z, slot=ints([5, slots - 1]), state_in=pool, state_out=pool)
    assert bool((y == z).all()) and bool((pool[[5, slots - 1]] == out).all())


def test_norm_rows_far_apart():
    x = torch.randn((40, 64), device="cuda").bfloat16()
    far = far_rows(40, 64, FAR // 39 + 8).copy_(x)
    for groups, shape in ((4, (40, 64)), (4, (2, 20, 64))):
        y, z = torch.empty_like(x), far_rows(40, 64, FAR // 39 + 8)
        fcm.group_norm(x.view(shape), y.view(shape), groups)
        strides = (z.stride(0), 1) if len(shape) == 2 else (20 * z.stride(0), z.stride(0), 1)
        fcm.group_norm(far.as_strided(shape, strides), z.as_strided(shape, strides), groups)
        assert bool((y == z).all())


def test_norm_of_a_map_past_32_bits():
    """2^31 and some elements in one sample, whose clusters leave their sums in y."""
    n = FAR // 64 + 1000
    x = torch.empty((1, n, 64), dtype=torch.bfloat16, device="cuda").normal_(2.0, 3.0)
    y = torch.empty_like(x)
    fcm.group_norm(x, y, 8)
    for g in range(0, 8, 3):
        v = x[0, :, 8 * g:8 * g + 8]
        mean = sum(float(p.double().sum()) for p in v.split(1 << 22)) / (8 * n)
        var = sum(float((p.double() - mean).square().sum()) for p in v.split(1 << 22)) / (8 * n)
        for at in (slice(0, 300), slice(n - 300, n)):
            want = (v[at].double() - mean) / (var + 1e-5) ** 0.5
            off = (y[0, at, 8 * g:8 * g + 8].double() - want).abs()
            # a rounding of the result; sums of 2^24 values in 32 bits, some 2^12 a thread: 2^-12 of the spread at most
            assert bool((off <= 2.0 ** -8 * want.abs() + 2.0 ** -11).all())


def test_mx4_rows_far_apart():
    x = torch.randn((9, 96), device="cuda").bfloat16()
    far, back = far_rows(9, 96, FAR // 8 + 8).copy_(x), far_rows(9, 96, FAR // 8 + 8)
    q, s, q2, s2 = (torch.empty((9, n), dtype=torch.uint8, device="cuda") for n in (48, 3, 48, 3))
    fcm.mx4_quantize(x, q, s)
    fcm.mx4_quantize(far, q2, s2)
    assert bool((q == q2).all()) and bool((s == s2).all())
    y = torch.empty_like(x)
    fcm.mx4_dequantize(q, s, y)
    fcm.mx4_dequantize(q, s, back)
    assert bool((y == back).all())
    near, wide = torch.empty((9, 50), device="cuda"), far_rows(9, 50, FAR // 8 + 8, torch.float32)
    w, ws = torch.randint(0, 256, (50, 48), dtype=torch.uint8, device="cuda"), torch.full((50, 3), 127, dtype=torch.uint8, device="cuda")
    fcm.mx4_matmul(q, s, w, ws, near)
    fcm.mx4_matmul(q, s, w, ws, wide)
    assert bool((near == wide).all())


def test_mx4_weights_past_32_bits():
    """Weights of 2^32 values, the last rows' bytes past 2^31."""
    out, k = FAR // 4096 + 200, 8192
    w = torch.randint(0, 256, (out, k // 2), dtype=torch.uint8, device="cuda")
    ws = torch.randint(120, 130, (out, k // 32), dtype=torch.uint8, device="cuda")
    xq, xs = w[:3].clone(), ws[:3].clone()
    y = torch.empty((3, out), device="cuda")
    fcm.mx4_matmul(xq, xs, w, ws, y)
    tail = torch.empty((3, 200), device="cuda")
    fcm.mx4_matmul(xq, xs, w[-200:].contiguous(), ws[-200:].contiguous(), tail)
    widened = [ref.mx4_values(ref.unpack(q.cpu().numpy()), s.cpu().numpy().astype(np.int64)) for q, s in ((xq, xs), (w[-200:], ws[-200:]))]
    want, e = ref.mx4_matmul(*widened, None, None, "none", "f32")
    within(y[:, -200:], want, e, "y")
    within(tail, want, e, "y")


def test_calls_on_two_streams_at_once():
    """The same kernels on different data at the same time, large maps among them, whose sums wait in their outputs."""
    g = torch.Generator("cuda").manual_seed(3)
    maps = [torch.randn((1, 300 * 300, 128), generator=g, device="cuda").bfloat16() for _ in range(2)]
    q, k, v = ([torch.randn((2, 200, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2)] for _ in range(3))
    d = [torch.randn((2, 200, 2), generator=g, device="cuda").bfloat16() for _ in range(2)]
    rows = [torch.randn((300, 512), generator=g, device="cuda").bfloat16() for _ in range(2)]
    a = -torch.ones(2, device="cuda")

    def calls(i, stream=None):
        y, z = torch.empty_like(maps[i]), torch.empty_like(v[i])
        c, s = torch.empty((300, 256), dtype=torch.uint8, device="cuda"), torch.empty((300, 16), dtype=torch.uint8, device="cuda")
        p = torch.empty((300, 300), device="cuda")
        return [y, z, c, s, p], lambda: (
            fcm.group_norm(maps[i], y, 32, act="silu", stream=stream),
            fcm.gated_delta(q[i], k[i], v[i], d[i], a, d[i], z, stream=stream),
            fcm.mx4_quantize(rows[i], c, s, stream=stream), fcm.mx4_matmul(c, s, c, s, p, stream=stream))
    want = []
    for i in range(2):
        out, run = calls(i)
        run()
        want.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = [calls(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for _, run in made:
            run()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(bool((x == w).all()) for x, w in zip(made[i][0], want[i]))


@pytest.mark.parametrize("n,pixels,c,dtype,kernel,count", [
    (1, 90000, 128, torch.bfloat16, "norm_apply", 2), (1, 3000, 128, torch.bfloat16, "norm_maps", 1),
    (4000, 1, 256, torch.bfloat16, "norm_rows", 1), (1, 90000, 127, torch.bfloat16, "norm_apply", 2)])
def test_norm_kernels_by_size(n, pixels, c, dtype, kernel, count):
    x = torch.zeros((n, pixels, c), dtype=dtype, device="cuda")
    y = torch.empty_like(x)
    found = captured(lambda s: fcm.group_norm(x, y, 1 if c % 2 else 8, stream=s))
    assert len(found) == count and kernel in found[-1].name


@pytest.mark.parametrize("dtype,dk,length,kernel", [
    (torch.bfloat16, 128, 1, "delta_row"), (torch.bfloat16, 128, 15, "delta_row"), (torch.bfloat16, 128, 16, "delta_chunk"),
    (torch.float16, 64, 300, "delta_chunk"), (torch.float32, 64, 300, "delta_row"), (torch.bfloat16, 129, 300, "delta_row")])
def test_delta_kernels_by_type_and_length(dtype, dk, length, kernel):
    q, v, d = (torch.zeros((1, length, *s), dtype=dtype, device="cuda") for s in ((1, dk), (1, 32), (1,)))
    y = torch.empty_like(v)
    found = captured(lambda s: fcm.gated_delta(q, q, v, d, torch.zeros(1, device="cuda"), d, y, stream=s))
    assert len(found) == 1 and kernel in found[0].name


@pytest.mark.parametrize("m,tokens,split", [(1, 16, 2), (20, 32, 2), (50, 64, 2), (100, 128, 2)])
def test_mx4_shapes_by_tokens(m, tokens, split):
    q, s = torch.zeros((m, 512), dtype=torch.uint8, device="cuda"), torch.zeros((m, 32), dtype=torch.uint8, device="cuda")
    y = torch.empty((m, 128), device="cuda")
    w, ws = torch.zeros((128, 512), dtype=torch.uint8, device="cuda"), torch.zeros((128, 32), dtype=torch.uint8, device="cuda")
    found = captured(lambda st: fcm.mx4_matmul(q, s, w, ws, y, stream=st))
    assert len(found) == 1 and found[0].numbers == (tokens,) and found[0].cluster == split


def test_empty_rows_and_sequences():
    e = torch.empty
    fcm.group_norm(e((0, 16), device="cuda"), e((0, 16), device="cuda"), 4)
    fcm.group_norm(e((2, 0, 16), device="cuda"), e((2, 0, 16), device="cuda"), 4)
    fcm.mx4_quantize(e((0, 64), device="cuda"), e((0, 32), dtype=torch.uint8, device="cuda"), e((0, 2), dtype=torch.uint8, device="cuda"))
    state = torch.randn((2, 1, 8, 8), device="cuda")
    out = torch.zeros_like(state)
    for dtype in (torch.float32, torch.bfloat16):
        z = e((0, 1, 8), device="cuda", dtype=dtype)
        fcm.gated_delta(z, z, z, z[..., 0], torch.zeros(1, device="cuda"), z[..., 0], z, seq_start=ints([0, 0, 0]),
                        max_len=20, state_in=state, state_out=out)
        assert bool((out == state).all())
        out.zero_()
