"""The 4-bit product over more inputs than a layer usually has: nothing limits them but an int."""
import numpy as np
import pytest

import pointwise_conv_cnn_gb300 as fcm
import seq_reference as ref
from helpers import torch_dtype

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,out,k,group", [(1, 17, 32800, 128), (3, 40, 65536, 64), (9, 20, 65568, 128), (2, 5, 131072 + 32, 32),
                                           (5, 2435, 65536, 128), (12, 2435, 40000, 64)])
def test_many_inputs(m, out, k, group, dtype):
    g = np.random.default_rng(k)
    x = torch.from_numpy(g.standard_normal((m, k))).to(torch_dtype(dtype)).cuda()
    q = g.integers(0, 16, (out, k))
    qs = torch.from_numpy(g.uniform(0.5, 1.5, (out, -(-k // group))) / np.sqrt(k)).to(x.dtype).cuda()
    y = torch.empty((m, out), dtype=x.dtype, device="cuda")
    fcm.w4_matvec(x, torch.from_numpy(ref.pack_w4(q)).cuda(), qs, y, group)
    want, e = ref.w4_matvec(x.double().cpu().numpy(), q, qs.double().cpu().numpy(), group, None, None, "none", dtype)
    assert bool((np.abs(y.double().cpu().numpy() - want) <= e).all())


@pytest.mark.slow
@pytest.mark.parametrize("group", [32, 128])
def test_as_many_inputs_as_an_int_counts(group):
    """2^31 - 32 of them, small whole numbers: every sum is exact, and one product that is left out shows."""
    k, piece = 2 ** 31 - 32, 1 << 26
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.empty((1, k), dtype=torch.bfloat16, device="cuda")
    qw = torch.empty((1, k // 2), dtype=torch.uint8, device="cuda")
    total = 0
    for at in range(0, k, piece):
        n = min(piece, k - at)
        v = torch.randint(-1, 2, (n,), generator=g, device="cuda", dtype=torch.int8)
        q = torch.randint(0, 256, (n // 2,), generator=g, device="cuda", dtype=torch.uint8)
        x[0, at:at + n], qw[0, at // 2:(at + n) // 2] = v.bfloat16(), q
        w = torch.stack((q & 15, q >> 4), -1).flatten().to(torch.int16) - 8
        total += int((w * v).sum(dtype=torch.int64))
    qs = torch.ones((1, -(-k // group)), dtype=torch.bfloat16, device="cuda")
    assert abs(total) < 2 ** 24

    def off(by):   # the sum less what it should be, which 16 bits hold exactly where it is small
        y = torch.empty((1, 1), dtype=torch.bfloat16, device="cuda")
        fcm.w4_matvec(x, qw, qs, y, group, scale=torch.ones(1, device="cuda"), bias=torch.tensor([-float(by)], device="cuda"))
        return float(y)
    assert off(total) == 0.0
    last = int((qw[0, -1] >> 4).to(torch.int16) - 8) * int(x[0, -1])
    x[0, -1] = 1.0
    qw[0, -1] = (qw[0, -1] & 15) | 0xF0   # the last weight is 7
    assert off(total - last) == 7.0
