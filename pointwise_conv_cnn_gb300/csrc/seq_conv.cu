// seq_conv.cu -- causal depthwise convolution over sequences with its cached rows.
//
// y[i,d] = act(s[d] * sum_j w[d,j] * xx[i+j,d] + b[d]), xx = the k-1 cached rows, then x.
#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct ConvArgs {
    Seqs q;
    const void *x, *w;
    const float *s, *b;
    const void *state_in;
    void *y, *state_out;
    long long ld_x, ld_y;
    int c, k, act;
    int rows;      // output rows per thread
    int tiles;     // tiles of `rows` rows that cover max_len
    long long threads;
};

constexpr int kMaxTaps = 8;

// One thread: one channel, a.rows consecutive rows of one sequence.
template <typename T>
__global__ void __launch_bounds__(128) causal_conv_kernel(const ConvArgs a) {
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const long long id = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= a.threads) return;
    const int d = (int)(id % a.c);
    const long long rest = id / a.c;
    const int tile = (int)(rest % a.tiles), q = (int)(rest / a.tiles);
    long long start;
    int len;
    seq_rows(a.q, q, start, len);
    const int i0 = tile * a.rows, h = a.k - 1;
    const T *x = static_cast<const T *>(a.x) + d + start * a.ld_x;
    T *y = static_cast<T *>(a.y) + d + start * a.ld_y;
    const int row = h > 0 && (a.state_in || a.state_out) ? state_row(a.q, q) : -1;
    const size_t at = row < 0 ? 0 : (size_t)row * h * a.c + d;
    T old[kMaxTaps - 1];   // the cached rows, read before any of them is replaced
    for (int j = 0; j < kMaxTaps - 1; j++) {
        old[j] = Storage<T>::from_f(0.0f);
        if (j < h && row >= 0 && a.state_in && tile == 0)
            old[j] = static_cast<const T *>(a.state_in)[at + (size_t)j * a.c];
    }
    auto in = [&](int i) -> T {   // place i of the sequence; places before 0 are the cached rows
        if (i >= 0) return x[(long long)i * a.ld_x];
        T v = old[0];
        for (int j = 1; j < kMaxTaps - 1; j++)
            if (j == i + h) v = old[j];
        return v;
    };
    float w[kMaxTaps];
    for (int j = 0; j < kMaxTaps; j++)
        w[j] = j < a.k ? Storage<T>::to_f(static_cast<const T *>(a.w)[(size_t)d * a.k + j]) : 0.0f;
    const float s = a.s ? a.s[d] : 1.0f, b = a.b ? a.b[d] : 0.0f;
    for (int i = i0; i < min(len, i0 + a.rows); i++) {
        float acc = 0.0f;
        for (int j = 0; j < kMaxTaps; j++)
            if (j < a.k) acc = fmaf(w[j], Storage<T>::to_f(in(i + j - h)), acc);
        y[(long long)i * a.ld_y] = Storage<T>::from_f(act_seq(fmaf(s, acc, b), a.act));
    }
    if (tile == 0 && row >= 0 && a.state_out)
        for (int j = 0; j < h; j++)
            static_cast<T *>(a.state_out)[at + (size_t)j * a.c] = in(len - h + j);
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_causal_conv(const fcm_causal_conv_desc *desc, const void *x,
                                      const void *w, const float *s, const float *b,
                                      const void *state_in, void *y, void *state_out,
                                      void *stream) {
    FcmNvtxRange nvtx("fcm_causal_conv");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_causal_conv_desc d = *desc;
    if (d.c < 1) return fcm_fail(FCM_ERR_INVALID_ARG, "c %d", d.c);
    if (d.ksize < 1 || d.ksize > seq::kMaxTaps)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "ksize %d outside 1..%d", d.ksize, seq::kMaxTaps);
    if (d.dtype < FCM_F32 || d.dtype > FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d.dtype);
    if (d.act < FCM_ACT_NONE || d.act > FCM_ACT_SILU)
        return fcm_fail(FCM_ERR_INVALID_ARG, "activation code out of range");
    if (d.ksize == 1) state_in = state_out = nullptr;
    seq::ConvArgs a = {};
    fcm_status st;
    if ((st = seq::check_seqs(d.seqs, state_in || state_out, &a.q)) != FCM_OK ||
        (st = seq::check_ld(&d.ld_x, d.c, "ld_x")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_y, d.c, "ld_y")) != FCM_OK)
        return st;
    if (a.q.n_seq == 0) return FCM_OK;
    const size_t e = (size_t)fcm_dtype_bytes(d.dtype);
    const bool rows = a.q.tokens > 0;   // x and y may be NULL when there is no row
    if ((rows && (st = seq::check_dev_ptr(x, e, "x")) != FCM_OK) ||
        (rows && (st = seq::check_dev_ptr(y, e, "y")) != FCM_OK) ||
        (st = seq::check_dev_ptr(w, e, "w")) != FCM_OK ||
        (s && (st = seq::check_dev_ptr(s, 4, "s")) != FCM_OK) ||
        (b && (st = seq::check_dev_ptr(b, 4, "b")) != FCM_OK) ||
        (state_in && (st = seq::check_dev_ptr(state_in, e, "state_in")) != FCM_OK) ||
        (state_out && (st = seq::check_dev_ptr(state_out, e, "state_out")) != FCM_OK))
        return st;
    if (seq::rows_overlap(x, d.ld_x, d.c, y, d.ld_y, d.c, a.q.tokens, e))
        return fcm_fail(FCM_ERR_INVALID_ARG, "x and y overlap");
    const long long state_row = (long long)(d.ksize - 1) * d.c;
    if (state_in != state_out &&
        seq::rows_overlap(state_in, state_row, state_row, state_out, state_row, state_row, a.q.slots, e))
        return fcm_fail(FCM_ERR_INVALID_ARG, "state_in and state_out overlap without being the same");
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;

    a.x = x, a.w = w, a.s = s, a.b = b, a.state_in = state_in, a.y = y, a.state_out = state_out;
    a.ld_x = d.ld_x, a.ld_y = d.ld_y, a.c = d.c, a.k = d.ksize, a.act = d.act;
    a.rows = 16;
    a.tiles = a.q.max_len ? (a.q.max_len + a.rows - 1) / a.rows : 1;
    a.threads = (long long)a.q.n_seq * a.tiles * a.c;
    const long long blocks = (a.threads + 127) / 128;
    if (blocks > 0x7FFFFFFFLL) return fcm_fail(FCM_ERR_UNSUPPORTED, "more than 2^31 thread blocks");
    void (*kernel)(seq::ConvArgs) = d.dtype == FCM_F32   ? seq::causal_conv_kernel<float>
                                    : d.dtype == FCM_F16 ? seq::causal_conv_kernel<__half>
                                                         : seq::causal_conv_kernel<__nv_bfloat16>;
    const cudaError_t ce = seq::launch(kernel, dim3((unsigned)blocks), 128, 0,
                                       static_cast<cudaStream_t>(stream), a);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
