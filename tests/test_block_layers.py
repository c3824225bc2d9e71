"""The gated delta rule, group normalisation and microscaled 4-bit values on the CPU: the references
against independent formulations, the descriptors' layout, and every refusal, none of which needs a GPU."""
import ctypes
import os
import re

import numpy as np
import pytest

import block_reference as ref
import pointwise_conv_cnn_gb300 as fcm

torch = pytest.importorskip("torch")
HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "fcm.h")


# ------------------------------------------------------------------------------ the references
def test_delta_reference_recalls_what_it_was_told():
    """Orthonormal keys, steps of 1, no decay: a key's value is what was written last."""
    k = np.zeros((5, 1, 4))
    k[range(5), 0, [0, 1, 2, 3, 1]] = 1.0
    v = np.arange(10.0).reshape(5, 1, 2)
    q = np.roll(k, 0, 0)
    zero, one = np.zeros((5, 1)), np.ones((5, 1))
    y, _, state, _ = ref.gated_delta(q, k, v, zero, np.zeros(1), one, None, False, False, False, 1.0, [(0, 5)], None,
                                     None, 1, "f32")
    np.testing.assert_allclose(y, v)
    np.testing.assert_allclose(state[0, 0], [[0, 1], [8, 9], [4, 5], [6, 7]])


def test_delta_reference_is_a_sum_where_keys_do_not_meet():
    """With a tiny step the rule is the decayed sum of k v^T."""
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((3, 6, 2, 4))
    v = v[:, :, :3]
    G, b = -g.random((6, 2)), np.full((6, 2), 1e-9)
    y, _, state, _ = ref.gated_delta(q, k, v, G, np.ones(2), b, None, False, False, False, 1.0, [(0, 6)], None, None, 1, "f32")
    want = sum(1e-9 * np.exp(G[t + 1:].sum(0))[:, None, None] * k[t][:, :, None] * v[t][:, None, :] for t in range(6))
    np.testing.assert_allclose(state[0], want, rtol=1e-6)
    np.testing.assert_allclose(y[5], np.einsum("hk,hkv->hv", q[5], want), rtol=1e-5, atol=1e-15)


def test_delta_reference_continues_where_it_stopped():
    g = np.random.default_rng(1)
    q, k = g.standard_normal((2, 7, 2, 5))
    v, dt, b = g.standard_normal((7, 4, 3)), g.standard_normal((7, 4)), g.standard_normal((7, 4))
    a, bias = -g.random(4), g.standard_normal(4)

    def part(i, j, state):
        return ref.gated_delta(q[i:j], k[i:j], v[i:j], dt[i:j], a, b[i:j], bias, True, True, True, 0.4, [(0, j - i)], None,
                               state, 1, "f32")
    y, _, end, _ = part(0, 7, None)
    y0, _, mid, _ = part(0, 3, None)
    y1, _, last, _ = part(3, 7, mid)
    np.testing.assert_array_equal(np.concatenate([y0, y1]), y)
    np.testing.assert_array_equal(last, end)


@pytest.mark.parametrize("groups,act", [(1, "none"), (3, "relu"), (6, "silu")])
def test_norm_reference_against_torch(groups, act):
    g = np.random.default_rng(2)
    x, s, b, z = g.standard_normal((2, 7, 6)), g.standard_normal(6), g.standard_normal(6), g.standard_normal((2, 7, 6))
    y, _ = ref.group_norm(x, groups, s, b, 1e-5, act, z, False, "f32")
    want = torch.nn.functional.group_norm(torch.from_numpy(x).mT, groups, torch.from_numpy(s), torch.from_numpy(b), 1e-5).mT
    want = {"none": lambda t: t, "relu": torch.relu, "silu": torch.nn.functional.silu}[act](want)
    np.testing.assert_allclose(y, (want * torch.nn.functional.silu(torch.from_numpy(z))).numpy(), rtol=1e-10, atol=1e-12)


def test_norm_reference_without_a_mean():
    x = np.array([[[3.0, 4.0, 1.0, 1.0]]])
    y, _ = ref.group_norm(x, 2, None, None, 0.0, "none", None, True, "f32")
    np.testing.assert_allclose(y[0, 0], [3 / 12.5 ** 0.5, 4 / 12.5 ** 0.5, 1.0, 1.0])


def test_mx4_reference_by_hand():
    x = np.zeros((1, 64))
    x[0, :10] = [4.0, 5.0, 0.25, 0.75, -1.25, 2.5, -3.5, 7.9, 0.26, -0.0]
    x[0, 32:34] = [1.0, 2.0 ** -3]
    codes, scale = ref.mx4_quantize(x)
    assert scale.tolist() == [[127, 125]]
    # 5 is between 4 and 6: 4's code is even; 0.25 between 0 and 0.5: 0; 0.75: 1; 1.25: 1; 2.5: 2; 3.5: 4; 7.9: 6 at most
    assert codes[0, :10].tolist() == [6, 6, 0, 2, 8 + 2, 4, 8 + 6, 7, 1, 8]
    assert codes[0, 32:34].tolist() == [6, 1]
    values = ref.mx4_values(codes, scale)
    assert values[0, [0, 4, 7, 32, 33]].tolist() == [4.0, -1.0, 6.0, 1.0, 0.125]
    assert ref.pack(codes)[0, :2].tolist() == [6 + 16 * 6, 0 + 16 * 2]
    np.testing.assert_array_equal(ref.unpack(ref.pack(codes)), codes)


# ------------------------------------------------------------------------------ the descriptors
@pytest.mark.parametrize("name,mirror,size", [
    ("fcm_delta_desc", fcm.FcmDeltaDesc, 128), ("fcm_norm_desc", fcm.FcmNormDesc, 64),
    ("fcm_mx4_desc", fcm.FcmMx4Desc, 24), ("fcm_mx4_matmul_desc", fcm.FcmMx4MatmulDesc, 32)])
def test_mirrors_follow_the_header(name, mirror, size):
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n for decl in body.split(";") for n in re.findall(r"\*?(\w+)\s*(?:,|$)", decl.strip())]
    assert [f.rstrip("_") for f, _ in mirror._fields_] == names
    assert ctypes.sizeof(mirror) == size


# ------------------------------------------------------------------------------ refusals
P = 1 << 16   # a well aligned address that is never followed


def refused(status, call, *args):
    with pytest.raises(fcm.FcmError) as e:
        call(*args)
    assert e.value.status == status, str(e.value)
    assert len(str(e.value)) > 15


def delta_desc(**kw):
    seqs = dict(tokens=6, n_seq=2, max_len=3, slots=2)
    d = dict(heads=4, key_heads=2, dk=8, dv=16, dtype=1, softplus=1, sigmoid=1, normalize=1, scale=1.0)
    for k, v in kw.items():
        (seqs if k in ("tokens", "n_seq", "max_len", "slots", "seq_start", "slot") else d)[k] = v
    return fcm.FcmDeltaDesc(seqs=fcm.FcmSeqs(**seqs), **d)


DELTA = [i * P for i in range(1, 11)]   # q, k, v, dt, a, b, dt_bias, state_in, y, state_out


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=7), 1), (dict(n_seq=-1, tokens=-3), 1), (dict(slots=1), 1), (dict(slots=0), 1), (dict(slot=P + 2), 3),
    (dict(seq_start=P + 1), 3), (dict(tokens=1 << 31, n_seq=1, max_len=(1 << 31) - 1, seq_start=P), 2),
    (dict(heads=0), 1), (dict(key_heads=0), 1), (dict(key_heads=3), 1), (dict(dk=0), 1), (dict(dk=257), 2), (dict(dv=0), 1),
    (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(softplus=2), 1), (dict(sigmoid=-1), 1), (dict(normalize=2), 1),
    (dict(ld_q=15), 1), (dict(ld_k=15), 1), (dict(ld_v=63), 1), (dict(ld_dt=3), 1), (dict(ld_b=3), 1), (dict(ld_y=63), 1),
    (dict(heads=1 << 20, dv=1 << 10), 2)])
def test_delta_descriptors_refused(kw, status):
    refused(status, fcm.fcm_gated_delta, delta_desc(**kw), *DELTA)


@pytest.mark.parametrize("which,value,status", [
    (0, 0, 1), (1, 0, 1), (2, 0, 1), (3, 0, 1), (4, 0, 1), (5, 0, 1), (8, 0, 1), (0, P + 1, 3), (1, P + 1, 3), (2, P + 1, 3),
    (3, P + 1, 3), (4, P + 2, 3), (5, P + 1, 3), (6, P + 2, 3), (7, P + 2, 3), (8, P + 1, 3), (9, P + 2, 3), (8, P, 1),
    (8, 2 * P + 4, 1), (8, 3 * P, 1), (8, 4 * P, 1), (8, 6 * P, 1), (9, 8 * P + 16, 1)])
def test_delta_pointers_refused(which, value, status):
    args = list(DELTA)
    args[which] = value
    refused(status, fcm.fcm_gated_delta, delta_desc(), *args)


NORM = [i * P for i in range(1, 6)]   # x, s, b, z, y


def norm_desc(**kw):
    return fcm.FcmNormDesc(**{**dict(n=2, c=16, groups=4, dtype=1, act=0, rms=0, eps=1e-5, pixels=9), **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(pixels=-1), 1), (dict(c=0), 1), (dict(groups=0), 1), (dict(groups=3), 1), (dict(groups=32), 1),
    (dict(dtype=3), 2), (dict(act=4), 1), (dict(act=-1), 1), (dict(rms=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(pixels=1 << 31), 2), (dict(c=8193, groups=1), 2), (dict(n=(1 << 31) - 1), 2),
    (dict(ld_x=15), 1), (dict(ld_z=8), 1), (dict(ld_y=-16), 1)])
def test_norm_descriptors_refused(kw, status):
    refused(status, fcm.fcm_group_norm, norm_desc(**kw), *NORM)


@pytest.mark.parametrize("which,value,status", [
    (0, 0, 1), (4, 0, 1), (0, P + 1, 3), (1, P + 2, 3), (2, P + 2, 3), (3, P + 1, 3), (4, P + 1, 3), (4, P + 32, 1),
    (4, 4 * P, 1)])
def test_norm_pointers_refused(which, value, status):
    args = list(NORM)
    args[which] = value
    refused(status, fcm.fcm_group_norm, norm_desc(), *args)


def test_norm_in_place_needs_the_same_rows():
    refused(1, fcm.fcm_group_norm, norm_desc(ld_x=16, ld_y=32), P, 0, 0, 0, P)


@pytest.mark.parametrize("call", ["fcm_mx4_quantize", "fcm_mx4_dequantize"])
@pytest.mark.parametrize("kw,status", [(dict(m=-1), 1), (dict(in_=0), 1), (dict(in_=48), 2), (dict(dtype=3), 2), (dict(ld=63), 1)])
def test_mx4_descriptors_refused(call, kw, status):
    d = fcm.FcmMx4Desc(**{**dict(m=3, in_=64, dtype=1), **kw})
    refused(status, getattr(fcm, call), d, P, 2 * P, 3 * P)


@pytest.mark.parametrize("which,value,status", [
    (0, 0, 1), (1, 0, 1), (2, 0, 1), (0, P + 1, 3), (1, P + 2, 3), (1, P + 64, 1), (2, P + 3, 1), (2, 2 * P + 5, 1)])
def test_mx4_pointers_refused(which, value, status):
    d = fcm.FcmMx4Desc(m=3, in_=64, dtype=1)
    args = [P, 2 * P, 3 * P]
    args[which] = value
    refused(status, fcm.fcm_mx4_quantize, d, *args)
    refused(status, fcm.fcm_mx4_dequantize, d, args[1], args[2], args[0])


MATMUL = [P, 2 * P, 3 * P, 4 * P, 0, 0, 5 * P]   # xq, xs, wq, ws, s, b, y


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(out=0), 1), (dict(in_=0), 1), (dict(in_=48), 2), (dict(dtype=3), 2), (dict(act=4), 1),
    (dict(ld_y=4), 1)])
def test_mx4_matmul_descriptors_refused(kw, status):
    d = fcm.FcmMx4MatmulDesc(**{**dict(m=3, out=5, in_=64, dtype=1, act=0), **kw})
    refused(status, fcm.fcm_mx4_matmul, d, *MATMUL)


@pytest.mark.parametrize("which,value,status", [
    (0, 0, 1), (1, 0, 1), (2, 0, 1), (3, 0, 1), (6, 0, 1), (0, P + 8, 3), (2, P + 8, 3), (4, P + 2, 3), (5, P + 2, 3),
    (6, P + 1, 3), (6, P + 32, 1), (6, 2 * P, 1)])
def test_mx4_matmul_pointers_refused(which, value, status):
    args = list(MATMUL)
    args[which] = value
    refused(status, fcm.fcm_mx4_matmul, fcm.FcmMx4MatmulDesc(m=3, out=5, in_=64, dtype=1), *args)


def test_null_descriptors_refused():
    lib = fcm.load_library()
    assert lib.fcm_gated_delta(*[None] * 12) == 1
    assert lib.fcm_group_norm(*[None] * 7) == 1
    assert lib.fcm_mx4_quantize(*[None] * 5) == 1
    assert lib.fcm_mx4_dequantize(*[None] * 5) == 1
    assert lib.fcm_mx4_matmul(*[None] * 9) == 1


def test_nothing_to_do_is_no_error():
    fcm.fcm_gated_delta(delta_desc(n_seq=0, tokens=0), *[0] * 10)
    fcm.fcm_group_norm(norm_desc(n=0), *[0] * 5)
    fcm.fcm_group_norm(norm_desc(pixels=0), *[0] * 5)
    fcm.fcm_mx4_quantize(fcm.FcmMx4Desc(m=0, in_=64, dtype=1), 0, 0, 0)
    fcm.fcm_mx4_dequantize(fcm.FcmMx4Desc(m=0, in_=64, dtype=1), 0, 0, 0)
    fcm.fcm_mx4_matmul(fcm.FcmMx4MatmulDesc(m=0, out=5, in_=64, dtype=1), *[0] * 7)


def test_binding_refuses_what_only_it_can_see():
    z = torch.zeros
    q, v, dt, a = z(2, 3, 2, 8), z(2, 3, 4, 16), z(2, 3, 4), z(4)
    x, byte = z(2, 5, 8), torch.uint8
    ok = (q, q, v, dt, a, dt, v)

    def delta(i, t, **kw):
        args = list(ok)
        args[i] = t
        return lambda: fcm.gated_delta(*args, **kw)
    bad = [
        (delta(0, q), "CUDA tensor"),
        (delta(0, q.double()), "float64"),
        (delta(0, q[0]), "seq_start"),
        (delta(1, q[:, :2]), "k must"),
        (delta(1, q.half()), "k must"),
        (delta(2, v[0]), "v must"),
        (delta(2, z(2, 3, 16, 4).transpose(2, 3)), "lie together"),
        (delta(3, z(2, 3, 2)), "dt must"),
        (delta(4, z(2)), "a must"),
        (delta(4, a.half()), "a must"),
        (delta(5, z(2, 3, 5)), "b must"),
        (delta(6, z(2, 3, 4, 15)), "y must"),
        (delta(6, z(3, 2, 4, 16).transpose(0, 1)), "same distance"),
        (delta(0, q, dt_bias=z(3)), "dt_bias must"),
        (delta(0, q, state_in=z(2, 4, 16, 8)), "state_in must"),
        (delta(0, q, state_out=z(2, 4, 8, 16).half()), "state_out must"),
        (delta(0, q, slot=z(2)), "slot must"),
        (delta(0, q, scale="x"), "scale must"),
        (lambda: fcm.gated_delta(z(6, 2, 8), z(6, 2, 8), z(6, 4, 16), z(6, 4), a, z(6, 4), z(6, 4, 16),
                                 seq_start=z(2, dtype=torch.int64)), "seq_start must"),
        (lambda: fcm.group_norm(x, x, 2), "CUDA tensor"),
        (lambda: fcm.group_norm(z(8), z(8), 2), "samples, channels"),
        (lambda: fcm.group_norm(x, x, 3), "divide"),
        (lambda: fcm.group_norm(x, x, 0), "divide"),
        (lambda: fcm.group_norm(x, x, "a"), "groups must"),
        (lambda: fcm.group_norm(x, x, 2.5), "groups must"),
        (lambda: fcm.group_norm(x, x.half(), 2), "y must"),
        (lambda: fcm.group_norm(x, x[:, :4], 2), "y must"),
        (lambda: fcm.group_norm(x, x, 2, z=z(2, 5, 7)), "z must"),
        (lambda: fcm.group_norm(x, x, 2, scale=z(7)), "scale must"),
        (lambda: fcm.group_norm(x, x, 2, bias=z(8).half()), "bias must"),
        (lambda: fcm.group_norm(x, x, 2, act="gelu"), "gelu"),
        (lambda: fcm.group_norm(x, z(2, 8, 5).mT, 2), "lie together"),
        (lambda: fcm.group_norm(x, z(5, 2, 8).transpose(0, 1), 2), "same distance"),
        (lambda: fcm.group_norm(x, z(1, 1, 8).expand(2, 5, 8), 2), "same distance|overlap"),
        (lambda: fcm.mx4_quantize(z(2, 64), z(2, 32, dtype=byte), z(2, 2, dtype=byte)), "CUDA tensor"),
        (lambda: fcm.mx4_quantize(z(2, 48), z(2, 24, dtype=byte), z(2, 1, dtype=byte)), "multiple of 32"),
        (lambda: fcm.mx4_quantize(z(2, 64), z(2, 31, dtype=byte), z(2, 2, dtype=byte)), "q must"),
        (lambda: fcm.mx4_quantize(z(2, 64), z(2, 32, dtype=byte), z(2, 2)), "s must"),
        (lambda: fcm.mx4_dequantize(z(2, 32, dtype=byte), z(2, 3, dtype=byte), z(2, 64)), "s must"),
        (lambda: fcm.mx4_dequantize(z(2, 32, dtype=byte), z(2, 2, dtype=byte), z(2, 64).long()), "y is"),
        (lambda: fcm.mx4_matmul(z(2, 32, dtype=byte), z(2, 2, dtype=byte), z(5, 32, dtype=byte), z(5, 2, dtype=byte), z(2, 5)),
         "CUDA tensor"),
        (lambda: fcm.mx4_matmul(z(2, 24, dtype=byte), z(2, 1, dtype=byte), z(5, 24, dtype=byte), z(5, 1, dtype=byte), z(2, 5)),
         "multiple of 32"),
        (lambda: fcm.mx4_matmul(z(2, 32, dtype=byte), z(2, 2, dtype=byte), z(5, 48, dtype=byte), z(5, 2, dtype=byte), z(2, 5)),
         "wq must"),
        (lambda: fcm.mx4_matmul(z(2, 32, dtype=byte), z(2, 1, dtype=byte), z(5, 32, dtype=byte), z(5, 2, dtype=byte), z(2, 5)),
         "xs must"),
        (lambda: fcm.mx4_matmul(z(2, 32, dtype=byte), z(2, 2, dtype=byte), z(5, 32, dtype=byte), z(5, 2, dtype=byte), z(2, 6)),
         "y must"),
    ]
    for i, (call, match) in enumerate(bad):
        with pytest.raises(fcm.FcmError, match=match):
            call()
            raise AssertionError(f"case {i} was not refused")
