// mx4_matmul.cu -- pointwise layer whose rows and weights are both microscaled 4-bit.
//
//     y[t,o] = act(s[o] * sum_i x[t,i] * w[o,i] + b[o])
#include "mx4.cuh"
#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct Mx4MatmulArgs {
    const uint8_t *xq, *xs, *wq, *ws;
    const float *s, *b;
    void *y;
    long long ld_y;
    int m, out, in, act;
};

// 64 rows by 64 outputs a block, a block of 32 inputs at a time: both factors widened in shared memory, four by
// four sums a thread.
template <typename T> __global__ void __launch_bounds__(256) mx4_matmul_kernel(const Mx4MatmulArgs a) {
    __shared__ float xt[32][65], wt[32][65];
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int m0 = blockIdx.y * 64, o0 = blockIdx.x * 64;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, r = threadIdx.x / 4, part = threadIdx.x % 4;
    const int half = a.in / 2, groups = a.in / 32;
    float sum[4][4] = {};
    for (int g = 0; g < groups; g++) {
        const int xr = min(m0 + r, a.m - 1), wr = min(o0 + r, a.out - 1);
        const uint32_t x = reinterpret_cast<const uint32_t *>(a.xq + (size_t)xr * half)[g * 4 + part];
        const uint32_t w = reinterpret_cast<const uint32_t *>(a.wq + (size_t)wr * half)[g * 4 + part];
        const float xb = power_of(a.xs[(size_t)xr * groups + g]), wb = power_of(a.ws[(size_t)wr * groups + g]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            xt[part * 8 + i][r] = e2m1_value(x >> (4 * i)) * xb;
            wt[part * 8 + i][r] = e2m1_value(w >> (4 * i)) * wb;
        }
        __syncthreads();
#pragma unroll 8
        for (int i = 0; i < 32; i++)
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int k = 0; k < 4; k++) sum[j][k] = fmaf(xt[i][ty * 4 + j], wt[i][tx + 16 * k], sum[j][k]);
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int t = m0 + ty * 4 + j, o = o0 + tx + 16 * k;
            if (t < a.m && o < a.out)
                static_cast<T *>(a.y)[(long long)t * a.ld_y + o] = Storage<T>::from_f(
                    act_seq(fmaf(a.s ? a.s[o] : 1.0f, sum[j][k], a.b ? a.b[o] : 0.0f), a.act));
        }
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_mx4_matmul(const fcm_mx4_matmul_desc *desc, const void *xq, const void *xs, const void *wq,
                                     const void *ws, const float *s, const float *b, void *y, void *stream) {
    FcmNvtxRange nvtx("fcm_mx4_matmul");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_mx4_matmul_desc d = *desc;
    if (d.m < 0 || d.out < 1 || d.in < 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "m %d, out %d, in %d", d.m, d.out, d.in);
    if (d.in % 32) return fcm_fail(FCM_ERR_UNSUPPORTED, "in %d is not a multiple of 32", d.in);
    if (d.dtype < FCM_F32 || d.dtype > FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d.dtype);
    if (d.act < FCM_ACT_NONE || d.act > FCM_ACT_SILU)
        return fcm_fail(FCM_ERR_INVALID_ARG, "activation code out of range");
    fcm_status st;
    if ((st = seq::check_ld(&d.ld_y, d.out, "ld_y")) != FCM_OK) return st;
    if (d.m == 0) return FCM_OK;
    const size_t e = (size_t)fcm_dtype_bytes(d.dtype);
    if ((st = seq::check_dev_ptr(xq, 16, "xq")) != FCM_OK || (st = seq::check_dev_ptr(xs, 1, "xs")) != FCM_OK ||
        (st = seq::check_dev_ptr(wq, 16, "wq")) != FCM_OK || (st = seq::check_dev_ptr(ws, 1, "ws")) != FCM_OK ||
        (st = seq::check_dev_ptr(y, e, "y")) != FCM_OK || (s && (st = seq::check_dev_ptr(s, 4, "s")) != FCM_OK) ||
        (b && (st = seq::check_dev_ptr(b, 4, "b")) != FCM_OK))
        return st;
    const long long half = d.in / 2, groups = d.in / 32, ldb = d.ld_y * (long long)e, row = d.out * (long long)e;
    if (seq::rows_overlap(xq, half, half, y, ldb, row, d.m, 1) || seq::rows_overlap(xs, groups, groups, y, ldb, row, d.m, 1))
        return fcm_fail(FCM_ERR_INVALID_ARG, "xq or xs and y overlap");
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;
    const seq::Mx4MatmulArgs a = {static_cast<const uint8_t *>(xq), static_cast<const uint8_t *>(xs),
                                  static_cast<const uint8_t *>(wq), static_cast<const uint8_t *>(ws), s, b, y, d.ld_y,
                                  d.m, d.out, d.in, d.act};
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)((d.out + 63) / 64), (unsigned)((d.m + 63) / 64));
    if (grid.y > 65535) return fcm_fail(FCM_ERR_UNSUPPORTED, "m %d above %d", d.m, 64 * 65535);
    const cudaError_t ce = seq::launch(d.dtype == FCM_F32   ? seq::mx4_matmul_kernel<float>
                                       : d.dtype == FCM_F16 ? seq::mx4_matmul_kernel<__half>
                                                            : seq::mx4_matmul_kernel<__nv_bfloat16>,
                                       grid, 256, 0, cs, a);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
