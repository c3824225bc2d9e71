"""How near the gated delta rule's outputs come in chunks of rows, where terms cancel: what y is computed from
has two rounded parts of 8 bits, off by 2^-17 of a number at most (the first leaves 2^-8 of the number's power of two, the
second half a step of that, 2^-9 of it), so S^T q by 2^-17 of its terms' sum and P u, both of whose factors have two parts,
by 2^-16.  The cases' terms are whole numbers, or sums of few, whose own errors stay under a tenth of that."""
import numpy as np
import pytest

import pointwise_conv_cnn_gb300 as fcm
from test_gpu_seq_layers import dev

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("cuda")]


def call(q, k, v, b, dtype, scale, state):
    """Rows [tokens, 1, ..] through the rule as it is told: no decay, steps b, keys as they are."""
    d = [dev(t, dtype) for t in (q, k, v, b)]
    for t, (_, held) in zip((q, k, v, b), d):
        assert (held == t).all()   # each number is one of the type
    (q, _), (k, _), (v, _), (b, _) = d
    zero, y = torch.zeros_like(b), torch.empty_like(v)
    fcm.gated_delta(q[None], k[None], v[None], zero[None], torch.zeros(1, device="cuda"), b[None], y[None], softplus=False,
                    sigmoid=False, normalize=False, scale=scale, state_in=None if state is None else dev(state, "f32")[0])
    return y.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dk", [64, 128])
def test_states_and_queries(dk, dtype):
    """Pairs of state rows 3 s and s, queries 1 and -3: y is 0.  s has 16 bits, two parts of 8; 3 s, 18 bits, has not."""
    g = np.random.default_rng(1)
    tokens, dv = 40, 32
    s = np.arange(43693, 44700, 4)
    s = g.choice(s[3 * s % 1024 >= 512], (dk // 2, dv))
    state = np.stack([3 * s, s], 1).reshape(1, 1, dk, dv)
    q = np.tile([1.0, -3.0], (tokens, 1, dk // 2))
    k, v, b = np.zeros((tokens, 1, dk)), np.zeros((tokens, 1, dv)), np.zeros((tokens, 1))
    y = call(q, k, v, b, dtype, 1.0, state)
    terms = (6.0 * s).sum(0)
    assert (np.abs(y) <= 2.0 ** -17 * terms).all(), np.abs(y / terms).max()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("first,second,value,scale", [(157, 205, 225, 128 ** -0.5), (195, 179, 193, 1.4137), (143, 213, 155, 1.9),
                                                      (211, 133, 251, 0.61)])
def test_rows_of_a_chunk(first, second, value, scale, dtype):
    """15 pairs of rows with keys of their own: queries a and -b find b c and a c, of 16 bits, and y is 0.  What scale a and
    scale b are off by in 32 bits is within U of the terms, and sums of 128 products, 4 of them a term, within 256 U."""
    tokens, dk, dv = 32, 64, 32
    eye = np.eye(tokens, dk)[:, None]
    a, b, c = first / 128.0, second / 128.0, value / 128.0
    q, step, v = np.zeros((tokens, 1, dk)), np.zeros((tokens, 1)), np.zeros((tokens, 1, dv))
    q[31, 0, :30] = np.tile([a, -b], 15)
    step[:30, 0], v[:30] = np.tile([b, a], 15), c
    y = call(q, eye, v, step, dtype, scale, None)
    terms = 30.0 * scale * a * b * c
    assert (y[:31] == 0.0).all() and (np.abs(y[31]) <= (2.0 ** -16 + 257.0 * 2.0 ** -24) * terms).all(), np.abs(y[31] / terms).max()
