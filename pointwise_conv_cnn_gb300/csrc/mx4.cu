// mx4.cu -- microscaled 4-bit floating point: quantising rows in blocks of 32 that share a power of two, and
// widening them again.
#include "mx4.cuh"
#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct Mx4Args {
    const void *in;      // x, or q
    const uint8_t *sin;
    void *out;           // y, or q
    uint8_t *sout;
    long long ld, blocks;   // blocks of 32 values in all
    int per_row;            // of them in a row
    int vec;                // rows of x or y start at 16 bytes
    int dense;              // and follow one another
};

// Where block b of 32 begins among rows ld apart.
__device__ __forceinline__ long long place(const Mx4Args &a, long long b) {
    return a.dense ? b * 32 : b / a.per_row * a.ld + b % a.per_row * 32;
}

// Eight neighbouring values as stored; one by one where rows do not start at 16 bytes.
template <typename T> __device__ __forceinline__ Vec<T, 8> load8(const T *p, int vec) {
    Vec<T, 8> v;
    constexpr int N = 16 / sizeof(T);
    if (vec) {
#pragma unroll
        for (int i = 0; i < 8; i += N)
            *reinterpret_cast<Vec<T, N> *>(&v.e[i]) = *reinterpret_cast<const Vec<T, N> *>(p + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v.e[i] = p[i];
    }
    return v;
}

// Four lanes a block of 32 values, each eight of them: 16 bytes in (two-byte types), four out.  The largest
// magnitude goes by its bits, whose order is the magnitudes' with infinity and NaN above all numbers; the
// power is its exponent.  Multiplying by a power of two is exact here: where a small value leaves the normal
// numbers it is nearer to 0 than a quarter, and rounds to 0 as it would have.
//
// Bound by memory: 8192 x 8192 bf16, quantised and widened again, 340 MB in 59 us, 5.7 TB/s, 0.85 of a plain copy's rate.
// (A division to find each block's row, which rows that follow one another do not need, took a quarter of that.)
template <typename T, int U> __global__ void __launch_bounds__(256) mx4_quantize_kernel(const Mx4Args a) {
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int part = threadIdx.x % 4;
    const long long first = (long long)blockIdx.x * (64 * U) + threadIdx.x / 4;
    Vec<T, 8> x[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const long long b = min(first + 64 * u, a.blocks - 1);
        x[u] = load8(static_cast<const T *>(a.in) + place(a, b) + 8 * part, a.vec);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        float v[8];
        x[u].get(v);
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const bool number = top < 0x7F800000u;
        const int e = max((int)(top >> 23) - 2, 0);             // code of the power; 253 at most
        const float by = __uint_as_float((unsigned)(254 - e) << 23);   // 2^(127 - e), a normal number
        uint32_t q = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) q |= e2m1_pair(v[i] * by, v[i + 1] * by) << (4 * i);
        const long long b = first + 64 * u;
        if (b < a.blocks) {
            static_cast<uint32_t *>(a.out)[b * 4 + part] = number ? q : 0u;
            if (part == 0) a.sout[b] = number ? (uint8_t)e : (uint8_t)255;
        }
    }
}

// The same lanes the other way.
template <typename T, int U> __global__ void __launch_bounds__(256) mx4_dequantize_kernel(const Mx4Args a) {
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int part = threadIdx.x % 4;
    const long long first = (long long)blockIdx.x * (64 * U) + threadIdx.x / 4;
    uint32_t q[U];
    unsigned e[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const long long b = min(first + 64 * u, a.blocks - 1);
        q[u] = static_cast<const uint32_t *>(a.in)[b * 4 + part];
        e[u] = a.sin[b];
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const long long b = first + 64 * u;
        if (b >= a.blocks) continue;
        const float by = power_of(e[u]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 x = e2m1_values(q[u] >> (4 * i));
            v[i] = x.x * by, v[i + 1] = x.y * by;
        }
        T *to = static_cast<T *>(a.out) + place(a, b) + 8 * part;
        constexpr int N = 16 / sizeof(T);
        Vec<T, 8> y;
        y.put(v);
        if (a.vec) {
#pragma unroll
            for (int i = 0; i < 8; i += N) *reinterpret_cast<Vec<T, N> *>(to + i) = *reinterpret_cast<Vec<T, N> *>(&y.e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) to[i] = y.e[i];
        }
    }
}

// Checks shared by both directions; false: there is nothing to do, or *st says what is wrong.
static bool mx4_ready(const fcm_mx4_desc *desc, fcm_mx4_desc *d, const void *x, const void *q, const void *s, Mx4Args *a,
                      fcm_status *st) {
    *st = FCM_OK;
    if (!desc) {
        *st = fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
        return false;
    }
    *d = *desc;
    if (d->m < 0 || d->in < 1) *st = fcm_fail(FCM_ERR_INVALID_ARG, "m %d, in %d", d->m, d->in);
    else if (d->in % 32) *st = fcm_fail(FCM_ERR_UNSUPPORTED, "in %d is not a multiple of 32", d->in);
    else if (d->dtype < FCM_F32 || d->dtype > FCM_BF16)
        *st = fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d->dtype);
    else *st = check_ld(&d->ld, d->in, "ld");
    if (*st != FCM_OK || d->m == 0) return false;
    const size_t e = (size_t)fcm_dtype_bytes(d->dtype);
    if ((*st = check_dev_ptr(x, e, "x or y")) != FCM_OK || (*st = check_dev_ptr(q, 4, "q")) != FCM_OK ||
        (*st = check_dev_ptr(s, 1, "s")) != FCM_OK)
        return false;
    const long long half = d->in / 2, groups = d->in / 32;
    // the three as rows of bytes
    const long long ld = d->ld * (long long)e, row = d->in * (long long)e;
    const struct {
        const void *p;
        long long ld, row;
    } t[3] = {{x, ld, row}, {q, half, half}, {s, groups, groups}};
    for (int i = 0; i < 3; i++)
        for (int j = 0; j < i; j++)
            if (rows_overlap(t[i].p, t[i].ld, t[i].row, t[j].p, t[j].ld, t[j].row, d->m, 1)) {
                *st = fcm_fail(FCM_ERR_INVALID_ARG, "q, s and x or y overlap");
                return false;
            }
    if (groups * d->m > 1LL << 38) {
        *st = fcm_fail(FCM_ERR_UNSUPPORTED, "%d rows of %d values: above 2^43 in all", d->m, d->in);
        return false;
    }
    int sms;
    if ((*st = current_device(&sms)) != FCM_OK) return false;
    a->ld = d->ld, a->per_row = (int)groups, a->blocks = groups * d->m;
    a->vec = aligned16(x) && ld % 16 == 0, a->dense = d->ld == d->in;
    return true;
}

constexpr int kMx4Unroll = 4;   // blocks of a lane on their way; 8192 x 8192 quantised and widened with 1, 2, 4: 76, 63, 59 us
static dim3 mx4_grid(const Mx4Args &a) { return dim3((unsigned)((a.blocks + 64 * kMx4Unroll - 1) / (64 * kMx4Unroll))); }

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_mx4_quantize(const fcm_mx4_desc *desc, const void *x, void *q, void *s, void *stream) {
    FcmNvtxRange nvtx("fcm_mx4_quantize");
    fcm_mx4_desc d;
    seq::Mx4Args a = {};
    fcm_status st;
    if (!seq::mx4_ready(desc, &d, x, q, s, &a, &st)) return st;
    a.in = x, a.out = q, a.sout = static_cast<uint8_t *>(s);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    constexpr int U = seq::kMx4Unroll;
    const cudaError_t ce = seq::launch(d.dtype == FCM_F32   ? seq::mx4_quantize_kernel<float, U>
                                       : d.dtype == FCM_F16 ? seq::mx4_quantize_kernel<__half, U>
                                                            : seq::mx4_quantize_kernel<__nv_bfloat16, U>,
                                       seq::mx4_grid(a), 256, 0, cs, a);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}

extern "C" fcm_status fcm_mx4_dequantize(const fcm_mx4_desc *desc, const void *q, const void *s, void *y, void *stream) {
    FcmNvtxRange nvtx("fcm_mx4_dequantize");
    fcm_mx4_desc d;
    seq::Mx4Args a = {};
    fcm_status st;
    if (!seq::mx4_ready(desc, &d, y, q, s, &a, &st)) return st;
    a.in = q, a.sin = static_cast<const uint8_t *>(s), a.out = y;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    constexpr int U = seq::kMx4Unroll;
    const cudaError_t ce = seq::launch(d.dtype == FCM_F32   ? seq::mx4_dequantize_kernel<float, U>
                                       : d.dtype == FCM_F16 ? seq::mx4_dequantize_kernel<__half, U>
                                                            : seq::mx4_dequantize_kernel<__nv_bfloat16, U>,
                                       seq::mx4_grid(a), 256, 0, cs, a);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
