// tensor_calls.cpp -- argument marshalling from torch tensors to the C ABI's layers over sequences
// (include/fcm.h), for the package's functions that take tensors (causal_conv and those below it).  A single token's
// kernel takes two or three microseconds, checking a call's dozen tensors attribute by attribute
// in Python ten; here it is less than one.  Nothing is computed, allocated or kept.
#define PY_SSIZE_T_CLEAN
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <sstream>
#include <string>

#include "../../include/fcm.h"

namespace {

PyObject *g_error = nullptr;   // FcmError
decltype(&fcm_causal_conv) g_conv = nullptr;
decltype(&fcm_selective_scan) g_scan = nullptr;
decltype(&fcm_w4_matvec) g_w4 = nullptr;
decltype(&fcm_gated_delta) g_delta = nullptr;
decltype(&fcm_group_norm) g_norm = nullptr;
decltype(&fcm_mx4_quantize) g_mx4_quantize = nullptr;
decltype(&fcm_mx4_dequantize) g_mx4_dequantize = nullptr;
decltype(&fcm_mx4_matmul) g_mx4_matmul = nullptr;
decltype(&fcm_last_error) g_last_error = nullptr;

struct Refusal {
    int status;
    std::string message;
};

template <typename... A> [[noreturn]] void refuse(int status, const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    throw Refusal{status, s.str()};
}

std::string shape_of(c10::IntArrayRef s) {
    std::ostringstream o;
    o << '(';
    for (size_t i = 0; i < s.size(); i++) o << (i ? ", " : "") << s[i];
    o << ')';
    return o.str();
}

std::string described(const at::Tensor &t) {
    std::ostringstream o;
    o << c10::toString(t.scalar_type()) << " " << shape_of(t.sizes()) << " with strides "
      << shape_of(t.strides()) << " on " << t.device();
    return o.str();
}

const at::Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) refuse(FCM_ERR_INVALID_ARG, what, " must be a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) refuse(FCM_ERR_INVALID_ARG, what, " must be a strided tensor");
    return t;
}

const at::Tensor *optional_tensor(PyObject *o, const char *what) {
    return o == Py_None ? nullptr : &tensor(o, what);
}

int dtype_code(const at::Tensor &x, const char *what = "x") {
    switch (x.scalar_type()) {
    case at::kFloat: return FCM_F32;
    case at::kHalf: return FCM_F16;
    case at::kBFloat16: return FCM_BF16;
    default:
        refuse(FCM_ERR_UNSUPPORTED, what, " is torch.",
               x.scalar_type() == at::kDouble ? "float64" : c10::toString(x.scalar_type()),
               ": float32, float16, bfloat16 are supported");
    }
}

// Address of a contiguous tensor of this type and shape on x's device (none: NULL).
template <typename P = const void>
P *plain(const at::Tensor *t, const at::Tensor &x, at::ScalarType type, std::initializer_list<int64_t> shape,
         const char *what) {
    if (!t) return nullptr;
    const c10::IntArrayRef want(shape.begin(), shape.size());
    if (t->scalar_type() != type || t->sizes() != want || t->device() != x.device() || !t->is_contiguous())
        refuse(FCM_ERR_INVALID_ARG, what, " must be a contiguous ", c10::toString(type), " tensor of shape ",
               shape_of(want), " on x's device, not ", described(*t));
    return static_cast<P *>(t->data_ptr());
}

// Row distance of activations [*lead, *row], whose row is a block of c elements side by side: x's type
// and device, all rows the same distance apart.
int64_t rows(const at::Tensor &t, const at::Tensor &x, c10::IntArrayRef lead, std::initializer_list<int64_t> row,
             const char *what) {
    const auto size = t.sizes();
    const auto stride = t.strides();
    const size_t n = lead.size();
    bool fits = t.scalar_type() == x.scalar_type() && t.device() == x.device() && size.size() == n + row.size();
    for (size_t i = 0; fits && i < size.size(); i++) fits = size[i] == (i < n ? lead[i] : row.begin()[i - n]);
    if (!fits) {
        std::vector<int64_t> want(lead.begin(), lead.end());
        want.insert(want.end(), row.begin(), row.end());
        refuse(FCM_ERR_INVALID_ARG, what, " must be a ", c10::toString(x.scalar_type()), " tensor of shape ",
               shape_of(want), " on x's device, not ", described(t));
    }
    int64_t c = 1;
    bool empty = false, dense = true;
    for (size_t i = row.size(); i-- > 0;) {
        dense = dense && (size[n + i] == 1 || stride[n + i] == c);
        c *= size[n + i];
    }
    for (const int64_t v : lead) empty = empty || v == 0;
    if (empty) return c;
    if (!dense) refuse(FCM_ERR_INVALID_ARG, what, ": a row's elements must lie together, strides ", shape_of(stride));
    int64_t ld = c;
    if (lead[n - 1] > 1) {
        ld = stride[n - 1];
        if (n == 2 && lead[0] > 1 && stride[0] != lead[1] * ld)
            refuse(FCM_ERR_INVALID_ARG, what, ": rows must all be the same distance apart, strides ", shape_of(stride));
    } else if (lead[0] > 1) {
        ld = stride[0];
    }
    if (ld < c) refuse(FCM_ERR_INVALID_ARG, what, ": rows overlap, strides ", shape_of(stride));
    return ld;
}

int as_int(int64_t v, const char *what) {
    if (v < 0 || v > 0x7FFFFFFF) refuse(FCM_ERR_INVALID_ARG, what, " ", v);
    return (int)v;
}

int act_code(PyObject *o) {
    static const char *const names[] = {"none", "relu", "relu6", "silu"};   // by fcm_act
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    for (int i = 0; s && i < 4; i++)
        if (!std::strcmp(s, names[i])) return i;
    PyErr_Clear();
    refuse(FCM_ERR_INVALID_ARG, "activation ", s ? s : "must be a name", ": none, relu, relu6 or silu");
}

bool truth(PyObject *o, const char *what) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        refuse(FCM_ERR_INVALID_ARG, what, " must be true or false");
    }
    return v != 0;
}

float number(PyObject *o, const char *what) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(FCM_ERR_INVALID_ARG, what, " must be a number");
    }
    return (float)v;
}

// The sequences of x [sequences, length, row], or of x [tokens, row] with seq_start, whose rows have `row`
// dimensions.
fcm_seqs sequences(const at::Tensor &x, const at::Tensor *seq_start, PyObject *max_len, const at::Tensor *slot,
                   const at::Tensor *state, int row = 1, const char *what = "x", const char *dims = "channels") {
    fcm_seqs s = {};
    if (!seq_start) {
        if (x.dim() != 2 + row)
            refuse(FCM_ERR_INVALID_ARG, what, " must be [sequences, length, ", dims, "], or [tokens, ", dims, "] with seq_start");
        s.n_seq = as_int(x.size(0), "sequences"), s.max_len = as_int(x.size(1), "length");
        s.tokens = (long long)s.n_seq * s.max_len;
    } else {
        if (x.dim() != 1 + row) refuse(FCM_ERR_INVALID_ARG, what, " must be [tokens, ", dims, "] with seq_start");
        if (seq_start->dim() != 1 || seq_start->size(0) < 1)
            refuse(FCM_ERR_INVALID_ARG, "seq_start must have one element more than there are sequences");
        s.tokens = x.size(0);
        s.n_seq = as_int(seq_start->size(0) - 1, "sequences");
        long long longest = s.tokens;
        if (max_len != Py_None) {
            longest = PyLong_AsLongLong(max_len);
            if (longest == -1 && PyErr_Occurred()) {
                PyErr_Clear();
                refuse(FCM_ERR_INVALID_ARG, "max_len must be a whole number");
            }
        }
        s.max_len = as_int(longest, "max_len");
        s.seq_start = plain<const int>(seq_start, x, at::kInt, {s.n_seq + 1LL}, "seq_start");
    }
    s.slot = plain<const int>(slot, x, at::kInt, {s.n_seq}, "slot");
    if (state) s.slots = state->dim() ? as_int(state->size(0), "slots") : 0;
    return s;
}

// The stream given (its handle, or an object that has it as cuda_stream), or the current one; x must
// lie on the current device.
void *stream_of(const at::Tensor &x, PyObject *stream, const char *what = "x") {
    if (!x.is_cuda() || x.get_device() != c10::cuda::current_device())
        refuse(FCM_ERR_INVALID_ARG, what, " must be a CUDA tensor on the current device");
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *handle = PyObject_GetAttrString(stream, "cuda_stream");
    if (!handle) {
        PyErr_Clear();
        Py_INCREF(stream);
        handle = stream;
    }
    void *p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(FCM_ERR_INVALID_ARG, "stream must be a stream or its handle");
    }
    return p;
}

PyObject *raise(int status, const char *message) {
    PyObject *args = Py_BuildValue("(is)", status, message);
    if (args) {
        PyErr_SetObject(g_error, args);
        Py_DECREF(args);
    }
    return nullptr;
}

// Runs a call's checks and the call: a refusal or a failure becomes an FcmError, and no C++ exception
// leaves.
template <typename F> PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F call) {
    if (given != wanted || !g_error) return raise(FCM_ERR_INVALID_ARG, "internal: wrong number of arguments, or not bound");
    try {
        const int status = call();
        if (status != FCM_OK) return raise(status, g_last_error());
    } catch (const Refusal &r) {
        return raise(r.status, r.message.c_str());
    } catch (const std::exception &e) {
        return raise(FCM_ERR_CUDA, e.what());
    } catch (...) {
        return raise(FCM_ERR_CUDA, "unknown exception");
    }
    Py_RETURN_NONE;
}

// x, w, y, scale, bias, act, seq_start, max_len, slot, state_in, state_out, stream
PyObject *causal_conv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> int {
        const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &y = tensor(a[2], "y");
        const at::Tensor *in = optional_tensor(a[9], "state_in"), *out = optional_tensor(a[10], "state_out");
        fcm_causal_conv_desc d = {};
        d.dtype = dtype_code(x);
        d.seqs = sequences(x, optional_tensor(a[6], "seq_start"), a[7], optional_tensor(a[8], "slot"), in ? in : out);
        if (w.dim() != 2) refuse(FCM_ERR_INVALID_ARG, "w must be [channels, ksize]");
        const int64_t c = x.sizes().back(), k = w.size(1), slots = d.seqs.slots;
        const auto lead = x.sizes().slice(0, x.dim() - 1);
        d.c = as_int(c, "channels"), d.ksize = as_int(k, "ksize"), d.act = act_code(a[5]);
        d.ld_x = rows(x, x, lead, {c}, "x"), d.ld_y = rows(y, x, lead, {c}, "y");
        const at::ScalarType type = x.scalar_type();
        const void *wp = plain(&w, x, type, {c, k}, "w");
        const float *s = plain<const float>(optional_tensor(a[3], "scale"), x, at::kFloat, {c}, "scale");
        const float *b = plain<const float>(optional_tensor(a[4], "bias"), x, at::kFloat, {c}, "bias");
        const void *sin = plain(in, x, type, {slots, k - 1, c}, "state_in");
        void *sout = plain<void>(out, x, type, {slots, k - 1, c}, "state_out");
        return g_conv(&d, x.data_ptr(), wp, s, b, sin, y.data_ptr(), sout, stream_of(x, a[11]));
    });
}

// x, dt, a, b, c, y, skip, z, dt_bias, softplus, seq_start, max_len, slot, state_in, state_out, stream
PyObject *selective_scan(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return guarded(n_args, 16, [&]() -> int {
        const at::Tensor &x = tensor(a[0], "x"), &dt = tensor(a[1], "dt"), &av = tensor(a[2], "a");
        const at::Tensor &b = tensor(a[3], "b"), &c = tensor(a[4], "c"), &y = tensor(a[5], "y");
        const at::Tensor *z = optional_tensor(a[7], "z");
        const at::Tensor *in = optional_tensor(a[13], "state_in"), *out = optional_tensor(a[14], "state_out");
        fcm_scan_desc d = {};
        d.dtype = dtype_code(x);
        d.seqs = sequences(x, optional_tensor(a[10], "seq_start"), a[11], optional_tensor(a[12], "slot"), in ? in : out);
        if (av.dim() != 2) refuse(FCM_ERR_INVALID_ARG, "a must be [channels, states]");
        const int64_t ch = x.sizes().back(), n = av.size(1), slots = d.seqs.slots;
        const auto lead = x.sizes().slice(0, x.dim() - 1);
        d.c = as_int(ch, "channels"), d.n_state = as_int(n, "states");
        d.softplus = truth(a[9], "softplus");
        d.ld_x = rows(x, x, lead, {ch}, "x"), d.ld_dt = rows(dt, x, lead, {ch}, "dt");
        if (b.dim() == x.dim() + 1) {
            const int64_t g = b.size(-2);
            d.groups = as_int(g, "groups");
            d.ld_b = rows(b, x, lead, {g, n}, "b"), d.ld_c = rows(c, x, lead, {g, n}, "c");
        } else {
            d.groups = 1;
            d.ld_b = rows(b, x, lead, {n}, "b"), d.ld_c = rows(c, x, lead, {n}, "c");
        }
        if (z) d.ld_z = rows(*z, x, lead, {ch}, "z");
        d.ld_y = rows(y, x, lead, {ch}, "y");
        const float *ap = plain<const float>(&av, x, at::kFloat, {ch, n}, "a");
        const float *skip = plain<const float>(optional_tensor(a[6], "skip"), x, at::kFloat, {ch}, "skip");
        const float *bias = plain<const float>(optional_tensor(a[8], "dt_bias"), x, at::kFloat, {ch}, "dt_bias");
        const float *sin = plain<const float>(in, x, at::kFloat, {slots, ch, n}, "state_in");
        float *sout = plain<float>(out, x, at::kFloat, {slots, ch, n}, "state_out");
        return g_scan(&d, x.data_ptr(), dt.data_ptr(), ap, b.data_ptr(), c.data_ptr(), skip, z ? z->data_ptr() : nullptr,
                      bias, sin, y.data_ptr(), sout, stream_of(x, a[15]));
    });
}

// x, qw, qs, y, group, scale, bias, act, stream
PyObject *w4_matvec(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> int {
        const at::Tensor &x = tensor(a[0], "x"), &qw = tensor(a[1], "qw"), &qs = tensor(a[2], "qs"), &y = tensor(a[3], "y");
        fcm_w4_desc d = {};
        d.dtype = dtype_code(x);
        if (x.dim() != 2 || qw.dim() != 2) refuse(FCM_ERR_INVALID_ARG, "x must be [m, in] and qw [out, in / 2]");
        const int64_t k = x.size(1), o = qw.size(0);
        const long group = PyLong_AsLong(a[4]);
        PyErr_Clear();
        if (group != 32 && group != 64 && group != 128)
            refuse(FCM_ERR_UNSUPPORTED, "group ", group, ": 32, 64 and 128 are supported");
        if (k % 32) refuse(FCM_ERR_UNSUPPORTED, "in ", k, " is not a multiple of 32");
        const auto lead = x.sizes().slice(0, 1);
        d.m = as_int(x.size(0), "m"), d.out = as_int(o, "out"), d.in = as_int(k, "in"), d.group = (int)group;
        d.act = act_code(a[7]);
        d.ld_x = rows(x, x, lead, {k}, "x"), d.ld_y = rows(y, x, lead, {o}, "y");
        const void *qp = plain(&qw, x, at::kByte, {o, k / 2}, "qw");
        const void *sp = plain(&qs, x, x.scalar_type(), {o, (k + group - 1) / group}, "qs");
        const float *s = plain<const float>(optional_tensor(a[5], "scale"), x, at::kFloat, {o}, "scale");
        const float *b = plain<const float>(optional_tensor(a[6], "bias"), x, at::kFloat, {o}, "bias");
        return g_w4(&d, x.data_ptr(), qp, sp, s, b, y.data_ptr(), stream_of(x, a[8]));
    });
}

// q, k, v, dt, a, b, y, dt_bias, softplus, sigmoid, normalize, scale, seq_start, max_len, slot, state_in, state_out, stream
PyObject *gated_delta(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 18, [&]() -> int {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &dt = tensor(a[3], "dt");
        const at::Tensor &av = tensor(a[4], "a"), &b = tensor(a[5], "b"), &y = tensor(a[6], "y");
        const at::Tensor *in = optional_tensor(a[15], "state_in"), *out = optional_tensor(a[16], "state_out");
        fcm_delta_desc d = {};
        d.dtype = dtype_code(q, "q");
        d.seqs = sequences(q, optional_tensor(a[12], "seq_start"), a[13], optional_tensor(a[14], "slot"), in ? in : out, 2,
                           "q", "key heads, dk");
        if (v.dim() != q.dim()) refuse(FCM_ERR_INVALID_ARG, "v must be shaped as q is, with [heads, dv] at its end");
        const int64_t hk = q.size(-2), dk = q.size(-1), h = v.size(-2), dv = v.size(-1), slots = d.seqs.slots;
        const auto lead = q.sizes().slice(0, q.dim() - 2);
        d.key_heads = as_int(hk, "key heads"), d.dk = as_int(dk, "dk"), d.heads = as_int(h, "heads"), d.dv = as_int(dv, "dv");
        d.softplus = truth(a[8], "softplus"), d.sigmoid = truth(a[9], "sigmoid"), d.normalize = truth(a[10], "normalize");
        d.scale = a[11] == Py_None ? (float)(1.0 / std::sqrt((double)(dk ? dk : 1))) : number(a[11], "scale");
        d.ld_q = rows(q, q, lead, {hk, dk}, "q"), d.ld_k = rows(k, q, lead, {hk, dk}, "k");
        d.ld_v = rows(v, q, lead, {h, dv}, "v"), d.ld_dt = rows(dt, q, lead, {h}, "dt");
        d.ld_b = rows(b, q, lead, {h}, "b"), d.ld_y = rows(y, q, lead, {h, dv}, "y");
        const float *ap = plain<const float>(&av, q, at::kFloat, {h}, "a");
        const float *bias = plain<const float>(optional_tensor(a[7], "dt_bias"), q, at::kFloat, {h}, "dt_bias");
        const float *sin = plain<const float>(in, q, at::kFloat, {slots, h, dk, dv}, "state_in");
        float *sout = plain<float>(out, q, at::kFloat, {slots, h, dk, dv}, "state_out");
        return g_delta(&d, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), ap, b.data_ptr(), bias, sin, y.data_ptr(),
                       sout, stream_of(q, a[17], "q"));
    });
}

// The distance of all rows of activations [sample, .., channel] behind one another, as if they were [rows, c]:
// dimensions of one element say nothing, the others have to continue each other.
int64_t pixel_rows(const at::Tensor &t, const at::Tensor &x, const char *what) {
    if (t.scalar_type() != x.scalar_type() || t.device() != x.device() || t.sizes() != x.sizes())
        refuse(FCM_ERR_INVALID_ARG, what, " must be a ", c10::toString(x.scalar_type()), " tensor of shape ",
               shape_of(x.sizes()), " on x's device, not ", described(t));
    const auto size = t.sizes(), stride = t.strides();
    const int64_t c = size.back();
    if (t.numel() == 0) return c;
    if (c > 1 && stride.back() != 1)
        refuse(FCM_ERR_INVALID_ARG, what, ": a row's elements must lie together, strides ", shape_of(stride));
    int64_t ld = c, next = 0;   // next: the stride that the dimension before has to have
    bool any = false;
    for (size_t i = size.size() - 1; i-- > 0;) {
        if (size[i] == 1) continue;
        if (!any) ld = stride[i];
        else if (stride[i] != next)
            refuse(FCM_ERR_INVALID_ARG, what, ": rows must all be the same distance apart, strides ", shape_of(stride));
        next = stride[i] * size[i], any = true;
    }
    if (ld < c) refuse(FCM_ERR_INVALID_ARG, what, ": rows overlap, strides ", shape_of(stride));
    return ld;
}

// x, y, groups, scale, bias, eps, act, z, rms, stream
PyObject *group_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> int {
        const at::Tensor &x = tensor(a[0], "x"), &y = tensor(a[1], "y");
        const at::Tensor *z = optional_tensor(a[7], "z");
        fcm_norm_desc d = {};
        d.dtype = dtype_code(x);
        if (x.dim() < 2) refuse(FCM_ERR_INVALID_ARG, "x must be [samples, channels] or [samples, .., channels]");
        const int64_t c = x.sizes().back();
        d.n = as_int(x.size(0), "samples"), d.c = as_int(c, "channels"), d.pixels = 1;
        for (int64_t i = 1; i + 1 < x.dim(); i++) d.pixels *= x.size(i);
        const long groups = PyLong_AsLong(a[2]);
        if (groups == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse(FCM_ERR_INVALID_ARG, "groups must be a whole number");
        }
        if (groups < 1 || groups > c || c % groups)
            refuse(FCM_ERR_INVALID_ARG, groups, " groups do not divide ", c, " channels");
        d.groups = (int)groups, d.act = act_code(a[6]), d.rms = truth(a[8], "rms"), d.eps = number(a[5], "eps");
        d.ld_x = pixel_rows(x, x, "x"), d.ld_y = pixel_rows(y, x, "y");
        if (z) d.ld_z = pixel_rows(*z, x, "z");
        const float *s = plain<const float>(optional_tensor(a[3], "scale"), x, at::kFloat, {c}, "scale");
        const float *b = plain<const float>(optional_tensor(a[4], "bias"), x, at::kFloat, {c}, "bias");
        return g_norm(&d, x.data_ptr(), s, b, z ? z->data_ptr() : nullptr, y.data_ptr(), stream_of(x, a[9]));
    });
}

// x (or y), q, s of microscaled rows
fcm_mx4_desc mx4_rows(const at::Tensor &x, const at::Tensor &q, const at::Tensor &s, const char *what) {
    fcm_mx4_desc d = {};
    d.dtype = dtype_code(x, what);
    if (x.dim() != 2) refuse(FCM_ERR_INVALID_ARG, what, " must be [rows, in]");
    const int64_t m = x.size(0), k = x.size(1);
    if (k % 32) refuse(FCM_ERR_UNSUPPORTED, "in ", k, " is not a multiple of 32");
    d.m = as_int(m, "rows"), d.in = as_int(k, "in");
    d.ld = rows(x, x, x.sizes().slice(0, 1), {k}, what);
    plain(&q, x, at::kByte, {m, k / 2}, "q"), plain(&s, x, at::kByte, {m, k / 32}, "s");
    return d;
}

// x, q, s, stream
PyObject *mx4_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> int {
        const at::Tensor &x = tensor(a[0], "x"), &q = tensor(a[1], "q"), &s = tensor(a[2], "s");
        const fcm_mx4_desc d = mx4_rows(x, q, s, "x");
        return g_mx4_quantize(&d, x.data_ptr(), q.data_ptr(), s.data_ptr(), stream_of(x, a[3]));
    });
}

// q, s, y, stream
PyObject *mx4_dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> int {
        const at::Tensor &q = tensor(a[0], "q"), &s = tensor(a[1], "s"), &y = tensor(a[2], "y");
        const fcm_mx4_desc d = mx4_rows(y, q, s, "y");
        return g_mx4_dequantize(&d, q.data_ptr(), s.data_ptr(), y.data_ptr(), stream_of(y, a[3], "y"));
    });
}

// xq, xs, wq, ws, y, scale, bias, act, stream
PyObject *mx4_matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> int {
        const at::Tensor &xq = tensor(a[0], "xq"), &xs = tensor(a[1], "xs"), &wq = tensor(a[2], "wq"), &ws = tensor(a[3], "ws");
        const at::Tensor &y = tensor(a[4], "y");
        fcm_mx4_matmul_desc d = {};
        d.dtype = dtype_code(y, "y");
        if (xq.dim() != 2 || wq.dim() != 2) refuse(FCM_ERR_INVALID_ARG, "xq must be [m, in / 2] and wq [out, in / 2]");
        const int64_t m = xq.size(0), o = wq.size(0), k = 2 * xq.size(1);
        if (k % 32) refuse(FCM_ERR_UNSUPPORTED, "in ", k, " is not a multiple of 32");
        d.m = as_int(m, "m"), d.out = as_int(o, "out"), d.in = as_int(k, "in"), d.act = act_code(a[7]);
        const int64_t lead[1] = {m};
        d.ld_y = rows(y, y, lead, {o}, "y");
        const void *xp = plain(&xq, y, at::kByte, {m, k / 2}, "xq"), *xsp = plain(&xs, y, at::kByte, {m, k / 32}, "xs");
        const void *wp = plain(&wq, y, at::kByte, {o, k / 2}, "wq"), *wsp = plain(&ws, y, at::kByte, {o, k / 32}, "ws");
        const float *s = plain<const float>(optional_tensor(a[5], "scale"), y, at::kFloat, {o}, "scale");
        const float *b = plain<const float>(optional_tensor(a[6], "bias"), y, at::kFloat, {o}, "bias");
        return g_mx4_matmul(&d, xp, xsp, wp, wsp, s, b, y.data_ptr(), stream_of(y, a[8], "y"));
    });
}

// FcmError and the addresses of the library's entry points, once, before any call.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int kCalls = 9;
    void *p[kCalls] = {};
    if (n != kCalls + 1) return PyErr_Format(PyExc_TypeError, "bind takes the error class and %d addresses", kCalls);
    for (int i = 0; i < kCalls; i++) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a NULL address");
    }
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    g_conv = reinterpret_cast<decltype(g_conv)>(p[0]);
    g_scan = reinterpret_cast<decltype(g_scan)>(p[1]);
    g_w4 = reinterpret_cast<decltype(g_w4)>(p[2]);
    g_delta = reinterpret_cast<decltype(g_delta)>(p[3]);
    g_norm = reinterpret_cast<decltype(g_norm)>(p[4]);
    g_mx4_quantize = reinterpret_cast<decltype(g_mx4_quantize)>(p[5]);
    g_mx4_dequantize = reinterpret_cast<decltype(g_mx4_dequantize)>(p[6]);
    g_mx4_matmul = reinterpret_cast<decltype(g_mx4_matmul)>(p[7]);
    g_last_error = reinterpret_cast<decltype(g_last_error)>(p[8]);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(causal_conv), FAST(selective_scan), FAST(w4_matvec), FAST(gated_delta),
                         FAST(group_norm), FAST(mx4_quantize), FAST(mx4_dequantize), FAST(mx4_matmul),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls(void) { return PyModule_Create(&module); }
