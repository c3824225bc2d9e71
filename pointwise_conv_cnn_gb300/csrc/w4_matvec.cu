// w4_matvec.cu -- pointwise layer for a few tokens with 4-bit weights and group scales.
//
//     y[t,o] = act(s[o] * sum_k x[t,k] * qs[o,k/group] * (q[o,k] - 8) + b[o])
#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct W4Args {
    const void *x, *qw, *qs;
    const float *s, *b;
    void *y;
    long long ld_x, ld_y;
    int m, out, in, group, act;
};

// One warp: one output of up to 16 tokens; a lane takes 8 weights of every 256.
template <typename T>
__global__ void __launch_bounds__(128) w4_simple_kernel(const W4Args a) {
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int lane = threadIdx.x & 31, o = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (o >= a.out) return;
    const int groups = (a.in + a.group - 1) / a.group;
    for (int t = blockIdx.y * 16; t < min(a.m, (int)blockIdx.y * 16 + 16); t++) {
        const T *x = static_cast<const T *>(a.x) + (long long)t * a.ld_x;
        float acc = 0.0f;
        for (int k = lane * 8; k < a.in; k += 256) {
            const uint32_t q = *reinterpret_cast<const uint32_t *>(
                static_cast<const uint8_t *>(a.qw) + ((size_t)o * a.in + k) / 2);
            float sum = 0.0f;
            for (int j = 0; j < 8; j++)
                sum = fmaf(Storage<T>::to_f(x[k + j]), (float)((int)(q >> (4 * j) & 15) - 8), sum);
            acc = fmaf(sum, Storage<T>::to_f(static_cast<const T *>(a.qs)[(size_t)o * groups + k / a.group]), acc);
        }
        for (int i = 16; i; i >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, i);
        if (lane == 0)
            static_cast<T *>(a.y)[(long long)t * a.ld_y + o] = Storage<T>::from_f(
                act_seq(fmaf(a.s ? a.s[o] : 1.0f, acc, a.b ? a.b[o] : 0.0f), a.act));
    }
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_w4_matvec(const fcm_w4_desc *desc, const void *x, const void *qw,
                                    const void *qs, const float *s, const float *b, void *y,
                                    void *stream) {
    FcmNvtxRange nvtx("fcm_w4_matvec");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_w4_desc d = *desc;
    if (d.m < 0 || d.out < 1 || d.in < 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "m %d, out %d, in %d", d.m, d.out, d.in);
    if (d.in % 32) return fcm_fail(FCM_ERR_UNSUPPORTED, "in %d is not a multiple of 32", d.in);
    if (d.group != 32 && d.group != 64 && d.group != 128)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "group %d: 32, 64 and 128 are supported", d.group);
    if (d.dtype != FCM_F16 && d.dtype != FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f16 and bf16 are supported", d.dtype);
    if (d.act < FCM_ACT_NONE || d.act > FCM_ACT_SILU)
        return fcm_fail(FCM_ERR_INVALID_ARG, "activation code out of range");
    fcm_status st;
    if ((st = seq::check_ld(&d.ld_x, d.in, "ld_x")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_y, d.out, "ld_y")) != FCM_OK)
        return st;
    if (d.m == 0) return FCM_OK;
    if ((st = seq::check_dev_ptr(x, 2, "x")) != FCM_OK || (st = seq::check_dev_ptr(y, 2, "y")) != FCM_OK ||
        (st = seq::check_dev_ptr(qw, 16, "qw")) != FCM_OK || (st = seq::check_dev_ptr(qs, 2, "qs")) != FCM_OK ||
        (s && (st = seq::check_dev_ptr(s, 4, "s")) != FCM_OK) ||
        (b && (st = seq::check_dev_ptr(b, 4, "b")) != FCM_OK))
        return st;
    if (seq::rows_overlap(x, d.ld_x, d.in, y, d.ld_y, d.out, d.m, 2))
        return fcm_fail(FCM_ERR_INVALID_ARG, "x and y overlap");
    if (d.m > 16 * 65535) return fcm_fail(FCM_ERR_UNSUPPORTED, "m %d above %d", d.m, 16 * 65535);
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;

    const seq::W4Args a = {x, qw, qs, s, b, y, d.ld_x, d.ld_y, d.m, d.out, d.in, d.group, d.act};
    const dim3 grid((unsigned)((d.out + 3) / 4), (unsigned)((d.m + 15) / 16));
    const cudaError_t ce = seq::launch(d.dtype == FCM_F16 ? seq::w4_simple_kernel<__half>
                                                          : seq::w4_simple_kernel<__nv_bfloat16>,
                                       grid, 128, 0, static_cast<cudaStream_t>(stream), a);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
