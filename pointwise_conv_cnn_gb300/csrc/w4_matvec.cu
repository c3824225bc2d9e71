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
    int m, out, in, act;
    int units;   // groups of inputs
};

// A 16 x 8 x 16 product on the tensor cores: rows are outputs, columns tokens.
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes, or zeros; a predicate instead of a branch, behind which nothing could be under way.
__device__ __forceinline__ uint4 load_if(const void *p, bool yes) {
    uint4 v = make_uint4(0, 0, 0, 0);
    asm("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"((int)yes));
    return v;
}

// The values of bits [4j, 4j + 4) and [4j + 16, 4j + 20) of q, less 8, in two halves: the bits are
// put into the mantissa of 1024 (f16) or 128 (bf16), so that the difference is exact.  f16's
// mantissa has room for them four places up as well, which saves shifts: 1024 + 16 q is scaled back.
template <typename T> __device__ __forceinline__ uint32_t two_weights(uint32_t q, int j) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value) {
        const uint32_t s = j >= 2 ? q >> 8 : q;
        if (j % 2 == 0) {
            const uint32_t v = (s & 0x000F000Fu) | 0x64006400u, o = 0x64086408u;   // 1024 + q, 1032
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(o));
        } else {
            const uint32_t v = (s & 0x00F000F0u) | 0x64006400u, k = 0x2C002C00u, o = 0xD480D480u;   // 1/16, -72
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(k), "r"(o));
        }
    } else {
        const uint32_t v = ((q >> (4 * j)) & 0x000F000Fu) | 0x43004300u, o = 0x43084308u;   // 128 + q, 136
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(o));
    }
    return r;
}

// One block: 16 outputs of up to 8 * NT tokens; its warps share the inputs' groups.  A lane of row
// r = lane / 4 and quarter t = lane % 4 holds the weights of rows r and r + 8 in quarter t of a
// group, and the inputs of token r there.  The product's inner index may run in any order as
// long as both sides follow it: a 32-bit word of eight weights gives the pairs (0,4), (1,5),
// (2,6), (3,7) with a shift and a mask each, and the inputs are paired alike.  So weights go
// from memory to the tensor cores as whole numbers, without a detour, and a group's sum is
// scaled in 32 bits.  XV: x's rows are 16-byte aligned.  SV: four scales are loaded at once, since a
// load whose lanes read eight rows takes eight turns at the cache whatever it brings.
template <typename T, int G, int NT, bool XV, bool SV>
__global__ void __launch_bounds__(512, NT == 1 ? 2 : 1) w4_kernel(const W4Args a) {
    constexpr int WORDS = G / 32;   // words per lane and group
    constexpr int UB = 128 / G;     // groups loaded at once
    extern __shared__ float red[];
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int r = lane >> 2, t = lane & 3, o0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
    // rows past the last output repeat it
    const int oa = min(o0 + r, a.out - 1), ob = min(o0 + r + 8, a.out - 1);
    const uint8_t *wa = static_cast<const uint8_t *>(a.qw) + (size_t)oa * (a.in / 2) + t * (G / 8);
    const uint8_t *wb = static_cast<const uint8_t *>(a.qw) + (size_t)ob * (a.in / 2) + t * (G / 8);
    const T *sa = static_cast<const T *>(a.qs) + (size_t)oa * a.units, *sb = static_cast<const T *>(a.qs) + (size_t)ob * a.units;
    // A column of the product is a token's alone.  Where there are fewer tokens, its inputs are not
    // read (the lanes of one token alone take a quarter of the cache's bandwidth that all take).
    const T *x[NT];
    bool token[NT];
#pragma unroll
    for (int i = 0; i < NT; i++) {
        token[i] = m0 + i * 8 + r < a.m;
        x[i] = static_cast<const T *>(a.x) + (long long)min(m0 + i * 8 + r, a.m - 1) * a.ld_x + t * (G / 4);
    }
    float sum[NT][4] = {};
    struct alignas(4 * WORDS) Words {
        uint32_t w[WORDS];
    };
    struct Inputs {
        uint4 v[NT][WORDS];
    };
    auto inputs = [&](int u) {
        Inputs in;
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int w = 0; w < WORDS; w++) {
                const T *p = x[i] + (size_t)u * G + w * 8;
                if (XV) {
                    in.v[i][w] = load_if(p, token[i]);
                } else {
                    const unsigned short *e = reinterpret_cast<const unsigned short *>(p);
                    in.v[i][w] = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                            e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
                }
            }
        return in;
    };
    auto group = [&](const Inputs &in, const Words &qa, const Words &qb, float fa, float fb) {
        constexpr int SUMS = WORDS >= 4 ? 2 : 1;   // a long group's products need not wait for each other
        float c[SUMS][NT][4] = {};
#pragma unroll
        for (int w = 0; w < WORDS; w++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t f[4] = {two_weights<T>(qa.w[w], 2 * h), two_weights<T>(qb.w[w], 2 * h),
                                       two_weights<T>(qa.w[w], 2 * h + 1), two_weights<T>(qb.w[w], 2 * h + 1)};
#pragma unroll
                for (int i = 0; i < NT; i++) {
                    const uint4 v = in.v[i][w];
                    const uint32_t lo = h ? v.y : v.x, hi = h ? v.w : v.z;
                    mma16816<T>(c[h % SUMS][i], f, __byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
                }
            }
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float v = SUMS == 2 ? c[0][i][j] + c[SUMS - 1][i][j] : c[0][i][j];
                sum[i][j] = fmaf(v, j < 2 ? fa : fb, sum[i][j]);
            }
    };
    constexpr int STEP = SV ? 4 : UB;   // groups a warp's share is a multiple of
    const int per = (a.units + warps * STEP - 1) / (warps * STEP) * STEP;
    const int u0 = min(a.units, warp * per), u1 = min(a.units, u0 + per);
    const int whole = min(u1, a.in / G);   // the last group may be short
    int u = u0;
    for (; u + STEP <= whole; u += STEP) {
        Vec<T, STEP> fa, fb;
        if (SV) {
            fa = *reinterpret_cast<const Vec<T, STEP> *>(sa + u);
            fb = *reinterpret_cast<const Vec<T, STEP> *>(sb + u);
        } else {
#pragma unroll
            for (int i = 0; i < STEP; i++) fa.e[i] = sa[u + i], fb.e[i] = sb[u + i];
        }
#pragma unroll
        for (int v = 0; v < STEP; v += UB) {
            Words qa[UB], qb[UB];
#pragma unroll
            for (int i = 0; i < UB; i++) {
                qa[i] = *reinterpret_cast<const Words *>(wa + (size_t)(u + v + i) * (G / 2));
                qb[i] = *reinterpret_cast<const Words *>(wb + (size_t)(u + v + i) * (G / 2));
            }
#pragma unroll
            for (int i = 0; i < UB; i++)
                group(inputs(u + v + i), qa[i], qb[i], Storage<T>::to_f(fa.e[v + i]), Storage<T>::to_f(fb.e[v + i]));
        }
    }
    for (; u < u1; u++) {
        const bool in = u * G + t * (G / 4) < a.in;   // a short group ends with a lane's quarter
        Words qa = {}, qb = {};
        Inputs v = {};                                // whose inputs past the end are zeros
        if (in) {
            qa = *reinterpret_cast<const Words *>(wa + (size_t)u * (G / 2));
            qb = *reinterpret_cast<const Words *>(wb + (size_t)u * (G / 2));
            v = inputs(u);
        }
        group(v, qa, qb, Storage<T>::to_f(sa[u]), Storage<T>::to_f(sb[u]));
    }
    // the warps' sums, in their order
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
        for (int j = 0; j < 4; j++)
            red[(warp * NT * 8 + i * 8 + 2 * t + (j & 1)) * 16 + r + (j >> 1) * 8] = sum[i][j];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 128; i += blockDim.x) {
        const int tok = m0 + i / 16, o = o0 + i % 16;
        if (tok >= a.m || o >= a.out) continue;
        float v = 0.0f;
        for (int w = 0; w < warps; w++) v += red[w * NT * 128 + i];
        static_cast<T *>(a.y)[(long long)tok * a.ld_y + o] = Storage<T>::from_f(
            act_seq(fmaf(a.s ? a.s[o] : 1.0f, v, a.b ? a.b[o] : 0.0f), a.act));
    }
}

template <typename T, int G>
static cudaError_t run_w4(const W4Args &a, int sms, cudaStream_t st) {
    const unsigned tiles = (unsigned)((a.out + 15) / 16), gy = (unsigned)((a.m + 15) / 16);
    // More warps share the inputs where the tiles leave SMs without a block, fewer where most SMs hold
    // two blocks and some a third.  Measured, us with 16, 8 and 4 warps: 4096 x 4096 (256 tiles) 4.3,
    // 5.4, -; 5003 x 4096 in groups of 32, 7 tokens (313) 8.4, 9.3, 7.5; 16384 x 8192 in groups
    // of 64 (1024) 25.2, 23.1, 26.8; 5120 x 5120, 16 tokens (320) 14.6, 12.1, 11.9.
    const unsigned long long blocks = (unsigned long long)tiles * gy;
    int warps = blocks < 2ull * sms ? 16 : blocks < 3ull * sms ? 4 : 8;
    while (warps > 4 && warps / 2 >= a.units) warps /= 2;
    const bool xv = aligned16(a.x) && a.ld_x % 8 == 0, wide = a.m > 8;
    // where that leaves no warp without work
    const bool sv = xv && !wide && a.units % 4 == 0 && a.units >= 4 * warps && reinterpret_cast<uintptr_t>(a.qs) % 8 == 0;
    void (*kernel)(W4Args) =
        wide ? (xv ? w4_kernel<T, G, 2, true, false> : w4_kernel<T, G, 2, false, false>)
             : (sv ? w4_kernel<T, G, 1, true, true> : xv ? w4_kernel<T, G, 1, true, false> : w4_kernel<T, G, 1, false, false>);
    return launch(kernel, dim3(tiles, gy), warps * 32, (size_t)warps * (wide ? 256 : 128) * 4, st, a);
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

    const seq::W4Args a = {x, qw, qs, s, b, y, d.ld_x, d.ld_y, d.m, d.out, d.in, d.act,
                           (d.in + d.group - 1) / d.group};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaError_t ce;
    if (d.dtype == FCM_F16)
        ce = d.group == 128  ? seq::run_w4<__half, 128>(a, sms, cs)
             : d.group == 64 ? seq::run_w4<__half, 64>(a, sms, cs)
                             : seq::run_w4<__half, 32>(a, sms, cs);
    else
        ce = d.group == 128  ? seq::run_w4<__nv_bfloat16, 128>(a, sms, cs)
             : d.group == 64 ? seq::run_w4<__nv_bfloat16, 64>(a, sms, cs)
                             : seq::run_w4<__nv_bfloat16, 32>(a, sms, cs);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
