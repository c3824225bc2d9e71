// seq_common.cuh -- what the layers over sequences share: the argument checks of fcm_seqs and of
// row-strided activations (host), each sequence's rows and state (device), and the launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fcm_device.cuh"
#include "fcm_internal.h"

namespace fcm {
namespace seq {

// fcm_seqs as the kernels take it.
struct Seqs {
    const int *seq_start;
    const int *slot;
    long long tokens;
    int n_seq, max_len, slots;
};

// Rows [start, start + len) of sequence q.  The bounds come from device memory the host has not
// seen: they are clamped to the tokens and to max_len, so no value leads outside the tensors.
__device__ __forceinline__ void seq_rows(const Seqs &s, int q, long long &start, int &len) {
    if (!s.seq_start) {
        start = (long long)q * s.max_len;
        len = s.max_len;
        return;
    }
    const long long b = s.seq_start[q], e = s.seq_start[q + 1];
    start = b < 0 ? 0 : b > s.tokens ? s.tokens : b;
    const long long end = e < start ? start : e > s.tokens ? s.tokens : e;
    len = (int)(end - start < s.max_len ? end - start : s.max_len);
}

// Row of sequence q in the state tensors, or -1 when it has none.
__device__ __forceinline__ int state_row(const Seqs &s, int q) {
    const int r = s.slot ? s.slot[q] : q;
    return r >= 0 && r < s.slots ? r : -1;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// v / (1 + e^-v).  Where the reciprocal of the sum is below the least normal number, from v = -87.34 down,
// the result is -0, its limit; no result that is lost is above 1.03e-36.  Keeping them (e^-v as a square of
// e^(-v/2), the sum held in range by 2^-32) cost the convolution of 16384 x 4096 1 us of 50.6, of 16384 x 4095
// 2.5 of 67.6, the scan of 4 x 2048 x 4096 2.3 of 175.7.
__device__ __forceinline__ float silu(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2(-kLog2e * v)));
    return v * r;
}

// The activations of fcm_act but silu.  NaN stays NaN, unlike in the fused modules, whose maximum drops it.
// (max.NaN and min.NaN in inline PTX cost the 4-bit product of one token with 1024 x 1024 2.20 us, these 2.03.)
__device__ __forceinline__ float clamp_act(float v, int act) {
    if (act == FCM_ACT_RELU) return v < 0.0f ? 0.0f : v;
    if (act == FCM_ACT_RELU6) return v < 0.0f ? 0.0f : v > 6.0f ? 6.0f : v;
    return v;
}
__device__ __forceinline__ float act_seq(float v, int act) {
    return act == FCM_ACT_SILU ? silu(v) : clamp_act(v, act);
}

// VEC consecutive elements, naturally aligned, as stored.  Plain loads: states are read and
// written by one kernel, and activations may just have been written by the kernel before.
template <typename T, int VEC> struct alignas(VEC * sizeof(T)) Vec {
    T e[VEC];
    __device__ __forceinline__ void get(float (&out)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; i++) out[i] = Storage<T>::to_f(e[i]);
    }
    __device__ __forceinline__ void put(const float (&in)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; i++) e[i] = Storage<T>::from_f(in[i]);
    }
};

// ------------------------------------------------------------------------------------- host
// Checks fcm_seqs; `state` says whether any state tensor was given.
fcm_status check_seqs(const fcm_seqs &s, bool state, Seqs *out);
// Row distance in elements (0: the row's own length).
fcm_status check_ld(long long *ld, long long row, const char *name);
// Pointer not NULL and aligned to `align` bytes.
fcm_status check_dev_ptr(const void *p, size_t align, const char *name);
// Whether row-strided tensors a and b, `rows` rows each, share a byte.  Column blocks of one wider
// tensor do not.
bool rows_overlap(const void *a, long long lda, long long ca, const void *b, long long ldb,
                  long long cb, long long rows, size_t esize);
// The current device's SM count; an error unless it is a compute capability 10.3 device.
fcm_status current_device(int *num_sms);

__host__ __device__ inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Launch with programmatic stream serialization allowed: the kernels wait for the previous grid
// (pdl_wait) before their first access to global memory.
template <typename A>
inline cudaError_t launch(void (*kernel)(A), dim3 grid, int threads, size_t smem, cudaStream_t st,
                          const A &a, int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace seq
}  // namespace fcm
