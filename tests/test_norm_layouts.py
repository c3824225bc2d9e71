"""Which layouts of activations group normalisation takes and refuses, on the CPU: what passes the check of
its rows is refused later, for not being on a GPU."""
import pytest

import pointwise_conv_cnn_gb300 as fcm

torch = pytest.importorskip("torch")

BROADCAST = [((2, 1, 8), (2, 5, 8)), ((4, 1, 1, 16), (4, 7, 7, 16)), ((2, 5, 1, 8), (2, 5, 3, 8)), ((2, 1, 3, 8), (2, 5, 3, 8)),
             ((1, 5, 8), (2, 5, 8)), ((1, 1, 8), (2, 5, 8)), ((1, 5, 1, 8), (2, 5, 3, 8)), ((2, 1, 1, 1, 8), (2, 2, 1, 3, 8)),
             ((1, 8), (3, 8)), ((3, 1, 1), (3, 5, 4)), ((1, 1), (3, 1))]


@pytest.mark.parametrize("held,shape", BROADCAST, ids=str)
@pytest.mark.parametrize("which", ["x", "y", "z"])
def test_broadcast_rows_are_refused(which, held, shape):
    """A dimension that is repeated has no rows of its own, whatever dimensions are around it."""
    t = {n: torch.zeros(shape) for n in "xyz"}
    t[which] = torch.zeros(held).expand(shape)
    with pytest.raises(fcm.FcmError, match=f": {which}: .*(same distance|overlap|lie together)"):
        fcm.group_norm(t["x"], t["y"], 1, z=t["z"])


@pytest.mark.parametrize("which", ["x", "y", "z"])
def test_rows_that_overlap_are_refused(which):
    t = {n: torch.zeros(2, 5, 8) for n in "xyz"}
    t[which] = torch.zeros(100).as_strided((2, 5, 8), (20, 4, 1))
    with pytest.raises(fcm.FcmError, match=f": {which}: rows overlap"):
        fcm.group_norm(t["x"], t["y"], 1, z=t["z"])


@pytest.mark.parametrize("shape,strides", [
    ((2, 5, 3, 8), (120, 24, 8, 1)), ((2, 5, 3, 8), (300, 60, 20, 1)), ((2, 5, 1, 8), (40, 8, 0, 1)), ((1, 5, 3, 8), (0, 24, 8, 1)),
    ((2, 1, 1, 8), (8, 0, 0, 1)), ((1, 1, 8), (0, 0, 1)), ((4, 8), (32, 1)), ((2, 0, 8), (0, 0, 1)), ((3, 5, 1), (5, 1, 0))])
def test_dimensions_of_one_element_say_nothing(shape, strides):
    t = [torch.zeros(1000).as_strided(shape, strides) for _ in range(3)]
    with pytest.raises(fcm.FcmError, match="CUDA tensor"):
        fcm.group_norm(t[0], t[1], 1, z=t[2])
