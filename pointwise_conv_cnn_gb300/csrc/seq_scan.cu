// seq_scan.cu -- selective scan over sequences.
//
//     h[d,n] = exp(D * a[d,n]) * h[d,n] + D * x[t,d] * bm[t,g,n],   D = softplus(dt[t,d] + dt_bias[d])
//     y[t,d] = (sum_n cm[t,g,n] * h[d,n] + skip[d] * x[t,d]) * silu(z[t,d])
#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct ScanArgs {
    Seqs q;
    const void *x, *dt, *bm, *cm, *z;
    const float *a, *skip, *dt_bias, *state_in;
    void *y;
    float *state_out;
    long long ld_x, ld_dt, ld_b, ld_c, ld_z, ld_y;
    int c, n, groups, softplus;
};

constexpr int kMaxState = 128;

// max(v, 0) + log(1 + e^-|v|).
__device__ __forceinline__ float softplus(float v) {
    return fmaxf(v, 0.0f) + log1pf(__expf(-fabsf(v)));
}

// One warp: one channel of one sequence, each lane up to four states.
template <typename T>
__global__ void __launch_bounds__(128) scan_simple_kernel(const ScanArgs a) {
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id >= (long long)a.q.n_seq * a.c) return;
    const int d = (int)(id % a.c), q = (int)(id / a.c), g = d / (a.c / a.groups);
    long long start;
    int len;
    seq_rows(a.q, q, start, len);
    const int row = a.state_in || a.state_out ? state_row(a.q, q) : -1;
    float av[4], h[4];
    for (int j = 0; j < 4; j++) {
        const int n = lane + 32 * j;
        av[j] = n < a.n ? a.a[(size_t)d * a.n + n] : 0.0f;
        h[j] = n < a.n && row >= 0 && a.state_in ? a.state_in[((size_t)row * a.c + d) * a.n + n] : 0.0f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.skip ? a.skip[d] : 0.0f;
    for (int i = 0; i < len; i++) {
        const long long t = start + i;
        const float u = Storage<T>::to_f(static_cast<const T *>(a.x)[t * a.ld_x + d]);
        float step = Storage<T>::to_f(static_cast<const T *>(a.dt)[t * a.ld_dt + d]) + bias;
        if (a.softplus) step = softplus(step);
        float o = 0.0f;
        for (int j = 0; j < 4; j++) {
            const int n = lane + 32 * j;
            if (n >= a.n) break;
            const float b = Storage<T>::to_f(static_cast<const T *>(a.bm)[t * a.ld_b + (long long)g * a.n + n]);
            const float c = Storage<T>::to_f(static_cast<const T *>(a.cm)[t * a.ld_c + (long long)g * a.n + n]);
            h[j] = fmaf(expf(step * av[j]), h[j], step * u * b);
            o = fmaf(c, h[j], o);
        }
        for (int m = 16; m; m >>= 1) o += __shfl_xor_sync(0xFFFFFFFFu, o, m);
        if (lane == 0) {
            if (a.skip) o = fmaf(skip, u, o);
            if (a.z) o *= silu(Storage<T>::to_f(static_cast<const T *>(a.z)[t * a.ld_z + d]));
            static_cast<T *>(a.y)[t * a.ld_y + d] = Storage<T>::from_f(o);
        }
    }
    if (row >= 0 && a.state_out)
        for (int j = 0; j < 4; j++)
            if (lane + 32 * j < a.n) a.state_out[((size_t)row * a.c + d) * a.n + lane + 32 * j] = h[j];
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_selective_scan(const fcm_scan_desc *desc, const void *x, const void *dt,
                                         const float *a, const void *bm, const void *cm,
                                         const float *skip, const void *z, const float *dt_bias,
                                         const float *state_in, void *y, float *state_out,
                                         void *stream) {
    FcmNvtxRange nvtx("fcm_selective_scan");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_scan_desc d = *desc;
    if (d.c < 1 || d.n_state < 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "c %d, n_state %d", d.c, d.n_state);
    if (d.n_state > seq::kMaxState)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "n_state %d above %d", d.n_state, seq::kMaxState);
    if (d.groups < 1 || d.c % d.groups)
        return fcm_fail(FCM_ERR_INVALID_ARG, "%d groups do not divide %d channels", d.groups, d.c);
    if (d.dtype < FCM_F32 || d.dtype > FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d.dtype);
    if (d.softplus != 0 && d.softplus != 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "softplus %d: 0 or 1", d.softplus);
    seq::ScanArgs k = {};
    const long long bc = (long long)d.groups * d.n_state;
    fcm_status st;
    if ((st = seq::check_seqs(d.seqs, state_in || state_out, &k.q)) != FCM_OK ||
        (st = seq::check_ld(&d.ld_x, d.c, "ld_x")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_dt, d.c, "ld_dt")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_b, bc, "ld_b")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_c, bc, "ld_c")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_z, d.c, "ld_z")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_y, d.c, "ld_y")) != FCM_OK)
        return st;
    if (k.q.n_seq == 0) return FCM_OK;
    const size_t e = (size_t)fcm_dtype_bytes(d.dtype);
    const long long rows = k.q.tokens;   // without rows the activations may be NULL
    if ((rows && ((st = seq::check_dev_ptr(x, e, "x")) != FCM_OK ||
                  (st = seq::check_dev_ptr(dt, e, "dt")) != FCM_OK ||
                  (st = seq::check_dev_ptr(bm, e, "bm")) != FCM_OK ||
                  (st = seq::check_dev_ptr(cm, e, "cm")) != FCM_OK ||
                  (st = seq::check_dev_ptr(y, e, "y")) != FCM_OK)) ||
        (z && (st = seq::check_dev_ptr(z, e, "z")) != FCM_OK) ||
        (st = seq::check_dev_ptr(a, 4, "a")) != FCM_OK ||
        (skip && (st = seq::check_dev_ptr(skip, 4, "skip")) != FCM_OK) ||
        (dt_bias && (st = seq::check_dev_ptr(dt_bias, 4, "dt_bias")) != FCM_OK) ||
        (state_in && (st = seq::check_dev_ptr(state_in, 4, "state_in")) != FCM_OK) ||
        (state_out && (st = seq::check_dev_ptr(state_out, 4, "state_out")) != FCM_OK))
        return st;
    const struct {
        const void *p;
        long long ld, cols;
        const char *name;
    } ins[] = {{x, d.ld_x, d.c, "x"}, {dt, d.ld_dt, d.c, "dt"}, {bm, d.ld_b, bc, "bm"},
               {cm, d.ld_c, bc, "cm"}, {z, d.ld_z, d.c, "z"}};
    for (const auto &in : ins)
        if (seq::rows_overlap(in.p, in.ld, in.cols, y, d.ld_y, d.c, rows, e))
            return fcm_fail(FCM_ERR_INVALID_ARG, "%s and y overlap", in.name);
    const long long state_row = (long long)d.c * d.n_state;
    if (state_in != state_out &&
        seq::rows_overlap(state_in, state_row, state_row, state_out, state_row, state_row, k.q.slots, 4))
        return fcm_fail(FCM_ERR_INVALID_ARG, "state_in and state_out overlap without being the same");
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;

    k.x = x, k.dt = dt, k.bm = bm, k.cm = cm, k.z = z, k.a = a, k.skip = skip, k.dt_bias = dt_bias;
    k.state_in = state_in, k.y = y, k.state_out = state_out;
    k.ld_x = d.ld_x, k.ld_dt = d.ld_dt, k.ld_b = d.ld_b, k.ld_c = d.ld_c, k.ld_z = d.ld_z, k.ld_y = d.ld_y;
    k.c = d.c, k.n = d.n_state, k.groups = d.groups, k.softplus = d.softplus;
    const long long blocks = ((long long)k.q.n_seq * k.c + 3) / 4;
    if (blocks > 0x7FFFFFFFLL) return fcm_fail(FCM_ERR_UNSUPPORTED, "more than 2^31 thread blocks");
    void (*kernel)(seq::ScanArgs) = d.dtype == FCM_F32   ? seq::scan_simple_kernel<float>
                                    : d.dtype == FCM_F16 ? seq::scan_simple_kernel<__half>
                                                         : seq::scan_simple_kernel<__nv_bfloat16>;
    const cudaError_t ce = seq::launch(kernel, dim3((unsigned)blocks), 128, 0,
                                       static_cast<cudaStream_t>(stream), k);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
