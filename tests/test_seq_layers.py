"""The layers over sequences on the CPU: the references against independent formulations, the
descriptors' layout, and every refusal, none of which needs a GPU."""
import ctypes
import os
import re

import numpy as np
import pytest

import pointwise_conv_cnn_gb300 as fcm
import seq_reference as ref

torch = pytest.importorskip("torch")
HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "fcm.h")


# ------------------------------------------------------------------------------ the references
def test_conv_reference_against_torch():
    g = np.random.default_rng(1)
    x, w, b = g.standard_normal((2, 9, 5)), g.standard_normal((5, 4)), g.standard_normal(5)
    y, _, state = ref.causal_conv(x.reshape(-1, 5), w, None, b, "silu", ref.bounds_of(2, 9), None,
                                  None, 2, "f32")
    xt = torch.nn.functional.pad(torch.from_numpy(x).transpose(1, 2), (3, 0))
    want = torch.nn.functional.silu(torch.nn.functional.conv1d(
        xt, torch.from_numpy(w)[:, None], torch.from_numpy(b), groups=5)).transpose(1, 2)
    np.testing.assert_allclose(y.reshape(2, 9, 5), want.numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(state, x[:, -3:])


def test_conv_reference_continues_where_it_stopped():
    g = np.random.default_rng(2)
    x, w = g.standard_normal((7, 3)), g.standard_normal((3, 4))
    whole, _, end = ref.causal_conv(x, w, None, None, "none", [(0, 7)], None, None, 1, "f32")
    a, _, mid = ref.causal_conv(x[:2], w, None, None, "none", [(0, 2)], None, None, 1, "f32")
    b, _, last = ref.causal_conv(x[2:], w, None, None, "none", [(0, 5)], None, mid, 1, "f32")
    np.testing.assert_array_equal(np.concatenate([a, b]), whole)
    np.testing.assert_array_equal(last, end)


def test_scan_reference_closed_forms():
    """Steps of 1: with a = 0 the state is a running sum; with a = -ln 2 and one input it halves."""
    ones = np.ones((6, 2))
    bm = np.ones((6, 1, 3))
    y, _, h, _ = ref.selective_scan(ones, ones, np.zeros((2, 3)), bm, bm, None, None, None, False,
                                    [(0, 6)], None, None, 1, "f32")
    np.testing.assert_allclose(y, 3.0 * np.arange(1, 7)[:, None] * ones)
    np.testing.assert_allclose(h, 6.0)
    x = np.zeros((6, 2))
    x[0] = 8.0
    y, _, h, _ = ref.selective_scan(x, ones, np.full((2, 3), -np.log(2.0)), bm, bm, np.ones(2), None,
                                    None, False, [(0, 6)], None, None, 1, "f32")
    np.testing.assert_allclose(y[:, 0], [32.0, 12.0, 6.0, 3.0, 1.5, 0.75])
    np.testing.assert_allclose(h, 0.25)


def test_w4_reference_by_hand():
    q = np.zeros((1, 32), np.int64)
    q[0, :4] = [15, 8, 0, 9]
    x = np.zeros((1, 32))
    x[0, :4] = [1.0, 10.0, 100.0, 1000.0]
    y, _ = ref.w4_matvec(x, q, np.array([[0.5]]), 32, np.array([2.0]), np.array([1.0]), "none", "f16")
    assert y[0, 0] == 2.0 * 0.5 * (7 + 0 - 800 + 1000) + 1.0
    assert ref.pack_w4(q)[0, :2].tolist() == [15 + 16 * 8, 0 + 16 * 9]


# ------------------------------------------------------------------------------ the descriptors
@pytest.mark.parametrize("name,mirror,size", [
    ("fcm_seqs", fcm.FcmSeqs, 40), ("fcm_causal_conv_desc", fcm.FcmCausalConvDesc, 72),
    ("fcm_scan_desc", fcm.FcmScanDesc, 112), ("fcm_w4_desc", fcm.FcmW4Desc, 40)])
def test_mirrors_follow_the_header(name, mirror, size):
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n for decl in body.split(";") for n in re.findall(r"\*?(\w+)\s*(?:,|$)", decl.strip())]
    assert [f.rstrip("_") for f, _ in mirror._fields_] == names
    assert ctypes.sizeof(mirror) == size


# ------------------------------------------------------------------------------ refusals
P = 4096   # a well aligned address that is never followed


def conv_desc(**kw):
    seqs = dict(tokens=6, n_seq=2, max_len=3, slots=2)
    d = dict(c=8, ksize=4, dtype=1, act=3, ld_x=0, ld_y=0)
    for k, v in kw.items():
        (seqs if k in ("tokens", "n_seq", "max_len", "slots", "seq_start", "slot") else d)[k] = v
    return fcm.FcmCausalConvDesc(seqs=fcm.FcmSeqs(**seqs), **d)


def scan_desc(**kw):
    seqs = dict(tokens=6, n_seq=2, max_len=3, slots=2)
    d = dict(c=8, n_state=4, groups=2, dtype=1, softplus=1)
    for k, v in kw.items():
        (seqs if k in ("tokens", "n_seq", "max_len", "slots", "seq_start", "slot") else d)[k] = v
    return fcm.FcmScanDesc(seqs=fcm.FcmSeqs(**seqs), **d)


BAD_SEQS = [(dict(tokens=7), 1), (dict(n_seq=-1, tokens=-3), 1), (dict(max_len=-1, tokens=-2), 1),
            (dict(slots=1), 1), (dict(slots=0), 1), (dict(slot=P + 2), 3), (dict(seq_start=P + 1), 3),
            (dict(tokens=1 << 31, n_seq=1, max_len=(1 << 31) - 1, seq_start=P), 2)]


def refused(status, call, *args):
    with pytest.raises(fcm.FcmError) as e:
        call(*args)
    assert e.value.status == status, str(e.value)
    assert len(str(e.value)) > 15


@pytest.mark.parametrize("kw,status", BAD_SEQS + [
    (dict(c=0), 1), (dict(ksize=0), 2), (dict(ksize=9), 2), (dict(dtype=3), 2), (dict(dtype=-1), 2),
    (dict(act=4), 1), (dict(act=-1), 1), (dict(ld_x=7), 1), (dict(ld_y=1), 1), (dict(ld_x=-8), 1)])
def test_conv_descriptors_refused(kw, status):
    refused(status, fcm.fcm_causal_conv, conv_desc(**kw), P, 2 * P, 0, 0, 3 * P, 4 * P, 5 * P)


@pytest.mark.parametrize("which,value,status", [
    (0, 0, 1), (1, 0, 1), (5, 0, 1), (0, P + 1, 3), (1, P + 1, 3), (2, P + 2, 3), (3, P + 2, 3),
    (4, P + 1, 3), (5, P + 1, 3), (6, P + 1, 3), (5, P + 2, 1), (5, P, 1), (6, 3 * P + 48, 1)])
def test_conv_pointers_refused(which, value, status):
    args = [P, 2 * P, 0, 0, 3 * P, 4 * P, 5 * P]
    args[which] = value
    refused(status, fcm.fcm_causal_conv, conv_desc(), *args)


@pytest.mark.parametrize("kw,status", BAD_SEQS + [
    (dict(c=0), 1), (dict(n_state=0), 1), (dict(n_state=129), 2), (dict(groups=0), 1),
    (dict(groups=3), 1), (dict(dtype=3), 2), (dict(softplus=2), 1), (dict(ld_x=7), 1), (dict(ld_dt=7), 1),
    (dict(ld_b=7), 1), (dict(ld_c=-1), 1), (dict(ld_z=1), 1), (dict(ld_y=2), 1)])
def test_scan_descriptors_refused(kw, status):
    refused(status, fcm.fcm_selective_scan, scan_desc(**kw), *[i * P for i in range(1, 12)])


@pytest.mark.parametrize("which,value,status", [
    (0, 0, 1), (1, 0, 1), (2, 0, 1), (3, 0, 1), (4, 0, 1), (9, 0, 1), (0, P + 1, 3), (2, P + 2, 3),
    (5, P + 2, 3), (6, P + 1, 3), (7, P + 2, 3), (8, P + 2, 3), (10, P + 2, 3), (9, P, 1),
    (9, 2 * P + 4, 1), (9, 4 * P, 1), (9, 5 * P, 1), (9, 7 * P, 1), (10, 9 * P + 16, 1)])
def test_scan_pointers_refused(which, value, status):
    args = [i * P for i in range(1, 12)]
    args[which] = value
    refused(status, fcm.fcm_selective_scan, scan_desc(), *args)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(out=0), 1), (dict(in_=0), 1), (dict(in_=48), 2), (dict(group=16), 2),
    (dict(group=256), 2), (dict(dtype=0), 2), (dict(dtype=3), 2), (dict(act=4), 1), (dict(ld_x=31), 1),
    (dict(ld_y=4), 1), (dict(m=1 << 30), 2)])
def test_w4_descriptors_refused(kw, status):
    d = dict(m=2, out=5, in_=64, group=32, dtype=1, act=0)
    refused(status, fcm.fcm_w4_matvec, fcm.FcmW4Desc(**{**d, **kw}),
            1 << 50, 2 * P, 3 * P, 0, 0, 1 << 20)


@pytest.mark.parametrize("which,value,status", [
    (0, 0, 1), (1, 0, 1), (2, 0, 1), (5, 0, 1), (0, P + 1, 3), (1, P + 8, 3), (2, P + 1, 3),
    (3, P + 2, 3), (4, P + 1, 3), (5, P + 1, 3), (5, P + 2, 1)])
def test_w4_pointers_refused(which, value, status):
    args = [P, 2 * P, 3 * P, 0, 0, 4 * P]
    args[which] = value
    refused(status, fcm.fcm_w4_matvec, fcm.FcmW4Desc(m=2, out=5, in_=64, group=32, dtype=1), *args)


def test_null_descriptors_refused():
    lib = fcm.load_library()
    assert lib.fcm_causal_conv(*[None] * 9) == 1
    assert lib.fcm_selective_scan(*[None] * 13) == 1
    assert lib.fcm_w4_matvec(*[None] * 8) == 1


def test_column_blocks_of_one_tensor_do_not_overlap():
    """x and y side by side in rows of 16: past the checks, and refused for want of a device."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these addresses must not be followed")
    d = conv_desc(ld_x=16, ld_y=16)
    refused(8, fcm.fcm_causal_conv, d, P, 2 * P, 0, 0, 0, P + 16, 0)
    refused(8, fcm.fcm_causal_conv, d, P + 16, 2 * P, 0, 0, 0, P, 0)
    refused(1, fcm.fcm_causal_conv, d, P, 2 * P, 0, 0, 0, P + 14, 0)
    refused(1, fcm.fcm_causal_conv, d, P + 18, 2 * P, 0, 0, 0, P, 0)


def test_nothing_to_do_is_no_error():
    """No sequence, or no row of x: nothing is launched and no device is needed."""
    fcm.fcm_causal_conv(conv_desc(n_seq=0, tokens=0), 0, 2 * P, 0, 0, 0, 0, 0)
    fcm.fcm_selective_scan(scan_desc(n_seq=0, tokens=0), *[0] * 11)
    fcm.fcm_w4_matvec(fcm.FcmW4Desc(m=0, out=5, in_=64, group=32, dtype=1), 0, 0, 0, 0, 0, 0)


def test_binding_refuses_what_only_it_can_see():
    x, y = torch.zeros(2, 3, 8), torch.zeros(2, 3, 8)
    w = torch.zeros(8, 4)
    bad = [
        (lambda: fcm.causal_conv(x, w, y), "CUDA tensor"),
        (lambda: fcm.causal_conv(x.double(), w, y), "float64"),
        (lambda: fcm.causal_conv(x[0], w, y), "seq_start"),
        (lambda: fcm.causal_conv(x, w.half(), y), "w must"),
        (lambda: fcm.causal_conv(x, w[:7], y), "w must"),
        (lambda: fcm.causal_conv(x, w, y[:1]), "y must"),
        (lambda: fcm.causal_conv(x, w, y.half()), "y must"),
        (lambda: fcm.causal_conv(x, w, torch.zeros(2, 8, 3).transpose(1, 2)), "lie together"),
        (lambda: fcm.causal_conv(x, w, torch.zeros(3, 2, 8).transpose(0, 1)), "same distance"),
        (lambda: fcm.causal_conv(x, w, torch.zeros(1, 1, 8).expand(2, 3, 8)), "same distance|overlap"),
        (lambda: fcm.causal_conv(x, w, y, bias=torch.zeros(7)), "bias must"),
        (lambda: fcm.causal_conv(x, w, y, scale=torch.zeros(8).half()), "scale must"),
        (lambda: fcm.causal_conv(x, w, y, act="gelu"), "gelu"),
        (lambda: fcm.causal_conv(x, w, y, state_in=torch.zeros(2, 4, 8)), "state_in must"),
        (lambda: fcm.causal_conv(x, w, y, state_in=torch.zeros(2, 3, 8), state_out=torch.zeros(3, 3, 8)),
         "state_out must"),
        (lambda: fcm.causal_conv(x, w, y, slot=torch.zeros(2)), "slot must"),
        (lambda: fcm.causal_conv(x[0], w, y[0], seq_start=torch.zeros(2, dtype=torch.int64)), "seq_start must"),
        (lambda: fcm.selective_scan(x, x, torch.zeros(8, 4), torch.zeros(2, 3, 4), torch.zeros(2, 3, 5), y), "c must"),
        (lambda: fcm.selective_scan(x, x, torch.zeros(7, 4), torch.zeros(2, 3, 4), torch.zeros(2, 3, 4), y), "a must"),
        (lambda: fcm.selective_scan(x, x, torch.zeros(8, 4), torch.zeros(2, 3, 2, 4), torch.zeros(2, 3, 1, 4), y), "c must"),
        (lambda: fcm.selective_scan(x, x[:, :2], torch.zeros(8, 4), torch.zeros(2, 3, 4), torch.zeros(2, 3, 4), y), "dt must"),
        (lambda: fcm.w4_matvec(torch.zeros(2, 48).half(), torch.zeros(5, 24).byte(), torch.zeros(5, 2).half(),
                               torch.zeros(2, 5).half(), 32), "multiple of 32"),
        (lambda: fcm.w4_matvec(torch.zeros(2, 64).half(), torch.zeros(5, 32).byte(), torch.zeros(5, 2).half(),
                               torch.zeros(2, 5).half(), 48), "group"),
        (lambda: fcm.w4_matvec(torch.zeros(2, 64).half(), torch.zeros(5, 16).byte(), torch.zeros(5, 2).half(),
                               torch.zeros(2, 5).half(), 32), "qw must"),
        (lambda: fcm.w4_matvec(torch.zeros(2, 64).half(), torch.zeros(5, 32).byte(), torch.zeros(5, 3).half(),
                               torch.zeros(2, 5).half(), 32), "qs must"),
    ]
    for call, match in bad:
        with pytest.raises(fcm.FcmError, match=match):
            call()


def test_modules_refuse_silu():
    with pytest.raises(fcm.FcmError) as e:
        fcm.fcm_plan_desc(fcm.make_desc(2, 8, 8, 16, 16, 3, 1, 1, act1="silu"))
    assert e.value.status == 1
