"""The example's block over many prompt lengths: what it keeps does not grow with them, and a shorter
prompt is the beginning of a longer one."""
import pytest

from test_gpu_ssm_block import example  # noqa: F401  (a fixture)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def test_lengths(example):  # noqa: F811
    block = example.SsmBlock()
    u = torch.randn((1, 600, 128), generator=torch.Generator("cpu").manual_seed(5)).to("cuda", torch.bfloat16)
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    whole = block(u, slot).double()
    for length in (17, 40, 63, 64, 65, 100, 127, 128, 191, 192, 193, 200, 255, 256, 300, 400, 511, 512, 513, 599):
        block.reset()
        got = block(u[:, :length].contiguous(), slot).double()
        off = (got - whole[:, :length]).norm() / whole[:, :length].norm()
        # each is off by the ten roundings that the block's own test counts
        assert off < 2 * 2.0 ** -8 * 10 ** 0.5, (length, float(off))
    kept = [len(p.modules) for p in (block.in_proj, block.x_proj, block.dt_proj, block.out_proj)]
    assert max(kept) <= 4, kept   # pieces of 64, 128, 256 and 512 rows
