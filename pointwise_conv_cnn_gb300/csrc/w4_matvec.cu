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

// 16 bytes, or zeros; a predicate instead of a branch, behind which nothing could be under way (a plain
// load under the condition: 7 tokens, 5003 x 4096 in groups of 32 8.2 us instead of 7.75).  The clobber
// keeps it behind pdl_wait: the kernel before may have written what it reads.
__device__ __forceinline__ uint4 load_if(const void *p, bool yes) {
    uint4 v = make_uint4(0, 0, 0, 0);
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"((int)yes) : "memory");
    return v;
}

// The values of bits [4j, 4j + 4) and [4j + 16, 4j + 20) of q, less 8, in two halves.  The long known
// conversion of small whole numbers without an instruction for it: the bits are put into the mantissa
// of a power of two whose last place is 1, 1024 (f16) or 128 (bf16), which the difference takes out exactly.  f16's
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

// One block: 16 * MT outputs of up to 8 * NT tokens; its warps share the inputs' groups.  A lane of row
// r = lane / 4 and quarter t = lane % 4 holds the weights of rows r, r + 8, .. in quarter t of a
// group, and the inputs of token r there.  The product's inner index may run in any order as
// long as both sides follow it: a 32-bit word of eight weights gives the pairs (0,4), (1,5),
// (2,6), (3,7) with a shift and a mask each, and the inputs are paired alike.  So weights go
// from memory to the tensor cores as whole numbers, without a detour, and a group's sum is
// scaled in 32 bits.  XV: x's rows are 16-byte aligned.  SV: four scales are loaded at once, since a
// load whose lanes read eight rows takes eight turns at the cache whatever it brings.
//
// The weights come from memory once: 20480 x 8192 in groups of 128, one token, 86.5 MB in 27.3 us, 3.2
// TB/s, 0.47 of a plain copy's rate.  What binds is the integer pipe that takes the weights apart (65 %
// busy: a shift, a mask and a difference each two weights) and, from eight tokens on, the cache's turns
// for the inputs (16 tokens 42.1 us, 0.77 of the cache's rate).  The warp-wide product is used since its
// factors come from registers, where the weights are; the larger ones of the tensor cores
// want them in shared memory, a detour of a store and a barrier for at most 16 columns, and the tensor cores
// are 20 % busy as it is.  Tried without gain: weights through a ring in shared memory (41 us), staged
// scales and inputs (38), one persistent block an SM (30 to 34), four tiles of outputs (33).
template <typename T, int G, int MT, int NT, bool XV, bool SV>
__global__ void __launch_bounds__(512, MT * NT == 1 ? 2 : 1) w4_kernel(const W4Args a) {
    constexpr int WORDS = G / 32;   // words per lane and group
    constexpr int UB = 128 / G;     // groups loaded at once
    constexpr int R = 2 * MT, OB = 16 * MT;   // rows of a lane, outputs of a block
    extern __shared__ float red[];
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int r = lane >> 2, t = lane & 3, m0 = blockIdx.y * 16;
    const unsigned o0 = blockIdx.x * OB;
    const uint8_t *wr[R];
    const T *sr[R];
#pragma unroll
    for (int i = 0; i < R; i++) {
        const unsigned o = min(o0 + r + 8 * i, (unsigned)a.out - 1);   // rows past the last output repeat it
        wr[i] = static_cast<const uint8_t *>(a.qw) + (size_t)o * (a.in / 2) + t * (G / 8);
        sr[i] = static_cast<const T *>(a.qs) + (size_t)o * a.units;
    }
    // A column of the product is a token's alone.  Where there are fewer tokens, its inputs are not
    // read (the lanes of one token alone take a quarter of the cache's bandwidth that all take).
    const T *x[NT];
    bool token[NT];
#pragma unroll
    for (int i = 0; i < NT; i++) {
        token[i] = m0 + i * 8 + r < a.m;
        x[i] = static_cast<const T *>(a.x) + (long long)min(m0 + i * 8 + r, a.m - 1) * a.ld_x + t * (G / 4);
    }
    float sum[MT][NT][4] = {};
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
    struct Weights {
        Words q[R];
    };
    auto weights = [&](int u) {
        Weights v;
#pragma unroll
        for (int i = 0; i < R; i++) v.q[i] = *reinterpret_cast<const Words *>(wr[i] + (size_t)u * (G / 2));
        return v;
    };
    auto group = [&](const Inputs &in, const Weights &q, const float (&f)[R]) {
        constexpr int SUMS = WORDS >= 4 && MT == 1 ? 2 : 1;   // a long group's products need not wait for each other
        float c[SUMS][MT][NT][4] = {};
#pragma unroll
        for (int w = 0; w < WORDS; w++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                uint32_t b[NT][2];
#pragma unroll
                for (int i = 0; i < NT; i++) {
                    const uint4 v = in.v[i][w];
                    const uint32_t lo = h ? v.y : v.x, hi = h ? v.w : v.z;
                    b[i][0] = __byte_perm(lo, hi, 0x5410), b[i][1] = __byte_perm(lo, hi, 0x7632);
                }
#pragma unroll
                for (int k = 0; k < MT; k++) {
                    const uint32_t qa = q.q[2 * k].w[w], qb = q.q[2 * k + 1].w[w];
                    const uint32_t m[4] = {two_weights<T>(qa, 2 * h), two_weights<T>(qb, 2 * h),
                                           two_weights<T>(qa, 2 * h + 1), two_weights<T>(qb, 2 * h + 1)};
#pragma unroll
                    for (int i = 0; i < NT; i++) mma16816<T>(c[h % SUMS][k][i], m, b[i][0], b[i][1]);
                }
            }
#pragma unroll
        for (int k = 0; k < MT; k++)
#pragma unroll
            for (int i = 0; i < NT; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float v = SUMS == 2 ? c[0][k][i][j] + c[SUMS - 1][k][i][j] : c[0][k][i][j];
                    sum[k][i][j] = fmaf(v, f[2 * k + j / 2], sum[k][i][j]);
                }
    };
    constexpr int STEP = SV ? 4 : UB;   // groups a warp's share is a multiple of
    const int per = (a.units + warps * STEP - 1) / (warps * STEP) * STEP;
    const int u0 = min(a.units, warp * per), u1 = min(a.units, u0 + per);
    const int whole = min(u1, a.in / G);   // the last group may be short
    int u = u0;
    for (; u + STEP <= whole; u += STEP) {
        Vec<T, STEP> f[R];
#pragma unroll
        for (int j = 0; j < R; j++) {
            if (SV) {
                f[j] = *reinterpret_cast<const Vec<T, STEP> *>(sr[j] + u);
            } else {
#pragma unroll
                for (int i = 0; i < STEP; i++) f[j].e[i] = sr[j][u + i];
            }
        }
#pragma unroll
        for (int v = 0; v < STEP; v += UB) {
            Weights q[UB];
#pragma unroll
            for (int i = 0; i < UB; i++) q[i] = weights(u + v + i);
#pragma unroll
            for (int i = 0; i < UB; i++) {
                float g[R];
#pragma unroll
                for (int j = 0; j < R; j++) g[j] = Storage<T>::to_f(f[j].e[v + i]);
                group(inputs(u + v + i), q[i], g);
            }
        }
    }
    for (; u < u1; u++) {
        const bool in = (unsigned)u * G + t * (G / 4) < (unsigned)a.in;   // a short group ends with a lane's quarter
        Weights q = {};
        Inputs v = {};                                // whose inputs past the end are zeros
        if (in) {
            q = weights(u);
            v = inputs(u);
        }
        float g[R];
#pragma unroll
        for (int j = 0; j < R; j++) g[j] = Storage<T>::to_f(sr[j][u]);
        group(v, q, g);
    }
    // the warps' sums, in their order
    constexpr int SUM = NT * 8 * OB;
#pragma unroll
    for (int k = 0; k < MT; k++)
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                red[warp * SUM + (i * 8 + 2 * t + (j & 1)) * OB + k * 16 + r + (j >> 1) * 8] = sum[k][i][j];
    __syncthreads();
    for (int i = threadIdx.x; i < SUM; i += blockDim.x) {
        const int tok = m0 + i / OB;
        const unsigned o = o0 + i % OB;
        if (tok >= a.m || o >= (unsigned)a.out) continue;
        float v = 0.0f;
        for (int w = 0; w < warps; w++) v += red[w * SUM + i];
        static_cast<T *>(a.y)[(long long)tok * a.ld_y + o] = Storage<T>::from_f(
            act_seq(fmaf(a.s ? a.s[o] : 1.0f, v, a.b ? a.b[o] : 0.0f), a.act));
    }
}

// One tile of 16 outputs a block or two.  Two halve the reads of the inputs, which with eight and
// more tokens cost more than the weights' (a warp's 16 rows of weights in a group of 128 are 16 turns
// at the cache, eight tokens' inputs 64), and their blocks need fewer rounds; one gives more
// blocks and shorter ones.  Measured, weights from memory, us with one and two: 20480 x 8192 in groups of 128, 1, 8,
// 16 tokens 27.8, 34.3, 61.9 and 27.3, 28.6, 42.4; 8192 x 8192 14.3, 15.1, 26.0 and 12.9, 13.2, 17.6; 4096 x 4096
// 5.3, 5.9, 8.2 and 5.6, 6.0, 7.1 (from the L2 4.8, 5.9, 8.2 and 4.6, 4.9, 7.0); 16384 x 4096 in groups of 64, 16
// tokens 23.7 and 19.1.  One tile: groups of 32 (5003 x 4096, 16 tokens 12.4 and 13.9), fewer blocks than half the
// SMs (2048 x 4096, 1, 8, 16 tokens 4.0, 4.4, 6.0 and 5.2, 5.4, 6.7), short sums (5120 x 1024, 16 tokens 4.4 and 4.7), and up to
// 8 tokens groups of 64, and scales that are not loaded by four (5120 x 5120, 1 token from the L2 7.1 and 7.7).
// Two tiles have 16 warps up to a block an SM, else 8.  16 tokens, us with 16, 8 and 4: 4096 x 4096 (128 blocks) 7.1, 8.5,
// 11.9; 5200 x 4096 in groups of 64 (163) 12.1, 10.6, 12.7; 8192 x 8192 (256) 20.0, 17.6, 21.8.
//
// More warps share the inputs where the tiles leave SMs without a block, fewer where every SM has several.
// Measured for one tile with weights that come from memory, us with 16, 8 and 4 warps, 18 output counts from 2000
// to 16384 each:
//   over 8 tokens, where a block of 16 warps has its SM to itself: 8 from the second block an SM on, but 4 from 2
//     to 2.4.  In groups of 32, 16 tokens: 2432 x 4096 (152 blocks) 6.6, 7.1, 9.6; 3600 x 4096 (225) 11.4, 9.3, 11.0; x 8192
//     17.8, 15.9, 18.7; 5600 x 4096 (350) 15.9, 14.4, 13.0; 6144 x 4096 (384) 16.0, 15.4, 19.1; x 2048 10.9, 9.4, 10.9;
//     13000 x 4096 (813) 29.8, 24.8, 27.5.
//   up to 8 tokens, fewer than two blocks an SM: 16.  3600 x 2048 in groups of 32, 8 tokens 4.7, 4.4, 5.1; 3600 x 4096 in
//     groups of 64, 1 token 5.6, 5.7, 7.9; x 8192 8.5, 9.5, 13.8.
//   two to three: 4, and 16 for long sums, where 4 do not keep enough loads under way.  Groups of 32, 1 token: 5003 x
//     2048 6.0, 5.5, 5.2; x 4096 8.8, 8.8, 8.4; x 8192 13.5, 15.3, 14.6.  Groups of 64: x 2048 5.5, 5.3, 5.1; x 8192 12.1, 14.1,
//     14.4; x 4096 7.4, 8.2, 8.4 from memory, but from the L2 6.3 with 16 and 6.1 with 4, 8 tokens 6.9 and 6.6.
//   more: 8.  16384 x 4096 in groups of 64, 1 token 15.7, 13.6, 14.7.
template <typename T, int G>
static cudaError_t run_w4(const W4Args &a, int sms, cudaStream_t st) {
    const bool xv = aligned16(a.x) && a.ld_x % 8 == 0, wide = a.m > 8;
    // Scales by four, where that leaves the warps' shares nearly alike.  Measured, weights from memory, us by four and one
    // by one: 5003 x 4096 in groups of 32 (128 of them, 4 warps), 1 and 7 tokens 8.4, 9.3 and 9.9, 10.7; 20480 x 8192 in
    // groups of 32 34.1 and 47.7; 5120 x 5120 in groups of 128 (40 of them, 4 warps) 10.5 and 9.5; 2048 x 4096 (32, 16
    // warps) 4.8 and 3.9.
    auto by_four = [&](int warps) {
        const long long per = (a.units + 4 * warps - 1) / (4 * warps) * 4;
        return xv && a.units % 4 == 0 && reinterpret_cast<uintptr_t>(a.qs) % 8 == 0 && per * warps * 8 <= a.units * 9ll;
    };
    const unsigned gy = (unsigned)((a.m + 15) / 16), pairs = ((unsigned)a.out + 31) / 32;
    const unsigned long long blocks2 = (unsigned long long)pairs * gy;
    if (xv && a.units >= 32 && 2 * blocks2 >= (unsigned long long)sms) {
        if constexpr (G >= 64)
            if (wide) {
                const int warps = blocks2 <= (unsigned long long)sms ? 16 : 8;
                return launch(by_four(warps) ? w4_kernel<T, G, 2, 2, true, true> : w4_kernel<T, G, 2, 2, true, false>,
                              dim3(pairs, gy), warps * 32, (size_t)warps * 512 * 4, st, a);
            }
        if constexpr (G == 128)
            if (!wide && by_four(8))
                return launch(w4_kernel<T, G, 2, 1, true, true>, dim3(pairs, gy), 256, (size_t)8 * 256 * 4, st, a);
    }
    const unsigned tiles = ((unsigned)a.out + 15) / 16;
    const unsigned long long blocks = (unsigned long long)tiles * gy;
    const unsigned long long n = (unsigned long long)sms;
    int warps = 8;
    if (blocks <= n || (!wide && blocks < 2 * n)) warps = 16;
    else if (wide && blocks >= 2 * n && 5 * blocks <= 12 * n) warps = 4;
    else if (!wide && blocks < 3 * n) warps = a.in < 8192 ? 4 : 16;
    while (warps > 4 && warps / 2 >= a.units) warps /= 2;
    void (*kernel)(W4Args) =
        wide ? (xv ? w4_kernel<T, G, 1, 2, true, false> : w4_kernel<T, G, 1, 2, false, false>)
             : (by_four(warps) ? w4_kernel<T, G, 1, 1, true, true>
                : xv           ? w4_kernel<T, G, 1, 1, true, false>
                               : w4_kernel<T, G, 1, 1, false, false>);
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
                           (d.in - 1) / d.group + 1};
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
