// delta_chunk.cuh -- the gated delta rule over prompts, 32 rows at a time on the tensor cores.
//
// Within a chunk, with c_i the sum of G up to row i, k and q as they enter the rule, and S before the chunk,
//     A_ij = B_i e^(c_i - c_j) k_i.k_j  (j < i),     T = (1 + A)^-1
//     x_i  = B_i (v_i - e^(c_i) S^T k_i),            u = T x
//     y_i  = scale (e^(c_i) S^T q_i + sum_{j <= i} e^(c_i - c_j) q_i.k_j u_j)
//     S'   = e^(c_last) S + sum_j e^(c_last - c_j) k_j u_j^T
// so that a chunk is a handful of small products.
#pragma once

#include "delta.cuh"

namespace fcm {
namespace seq {

template <int DK> struct DeltaChunk {
    static constexpr int C = 32;                      // rows of a chunk
    static constexpr int DS = DK / 32;                // warps that share 16 columns' states, 32 keys each
    static constexpr int STATE = 2 * DS, FRONT = 4;   // warps
    static constexpr int THREADS = 32 * (STATE + FRONT + 1);
    static constexpr int SLOTS = 3;
    static constexpr int KS = 2 * DK + 16;            // bytes of a row of keys: eight rows in different banks
    static constexpr int TS = 80;                     // of T and of the rows' products P
    static constexpr int VS = 80;                     // of values
    static constexpr int AS = 36;                     // floats of a row of A
    // a slot's parts, bytes
    static constexpr int Q = C * KS, V = 2 * C * KS, THI = V + C * VS, TLO = THI + C * TS, PHI = TLO + C * TS,
                         PLO = PHI + C * TS, A = PLO + C * TS, SC = A + C * AS * 4, SLOT = SC + 12 * C * 4;
    static constexpr int XCH = 2 * 2 * DS * 8 * 512;   // sums on their way between warps: [turn][16 columns][warp][16 bytes][lane]
    static constexpr int SMEM = SLOTS * SLOT + XCH;
};
// A slot's factors by row
enum { kBeta, kBetaReach, kQReach, kToEnd, kTDown, kPDown, kFk, kFq, kSumHi, kSumLo, kTotal };

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_half(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// The power of two that brings numbers of this largest magnitude (its bits) to 2^14 .. 2^15, inside f16's range, and
// its inverse.  Both are normal numbers; infinities and NaN stay what they are.
struct Power {
    float up, down;
    __device__ __forceinline__ explicit Power(uint32_t top) {
        const int f = min(max(268 - (int)(top >> 23), 1), 253);
        up = __uint_as_float((uint32_t)f << 23), down = __uint_as_float((uint32_t)(254 - f) << 23);
    }
};
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Two numbers in two 16-bit parts each: 22 bits of them.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h), lo = *reinterpret_cast<const uint32_t *>(&l);
}

// N tiles of 16 x 8 sums as the left factors of the next product, in two parts, each of a lane's two rows times a
// power of two that its four lanes agree on; `down` undoes it.  Tiles 2 i and 2 i + 1 are 16 inner places.
template <int N>
__device__ __forceinline__ void as_factor(const float (&c)[N][4], uint32_t (&hi)[N / 2][4], uint32_t (&lo)[N / 2][4], float (&down)[2]) {
    uint32_t top[2] = {};
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) top[e / 2] = max(top[e / 2], magnitude(c[i][e]));
    float up[2];
#pragma unroll
    for (int r = 0; r < 2; r++) {
        top[r] = max(top[r], __shfl_xor_sync(~0u, top[r], 1));
        top[r] = max(top[r], __shfl_xor_sync(~0u, top[r], 2));
        const Power p(top[r]);
        up[r] = p.up, down[r] = p.down;
    }
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int r = 0; r < 2; r++)
            split2(c[i][2 * r] * up[r], c[i][2 * r + 1] * up[r], hi[i / 2][i % 2 * 2 + r], lo[i / 2][i % 2 * 2 + r]);
}

// Eight neighbouring keys or queries of a row, zeros past the row's end.
template <typename T> __device__ __forceinline__ uint4 load_keys(const T *p, int e, int dk, bool live, bool vec) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!live || e >= dk) return v;
    if (vec) return *reinterpret_cast<const uint4 *>(p + e);
    unsigned short s[8];
#pragma unroll
    for (int i = 0; i < 8; i++) s[i] = e + i < dk ? reinterpret_cast<const unsigned short *>(p)[e + i] : (unsigned short)0;
    v.x = s[0] | (uint32_t)s[1] << 16, v.y = s[2] | (uint32_t)s[3] << 16;
    v.z = s[4] | (uint32_t)s[5] << 16, v.w = s[6] | (uint32_t)s[7] << 16;
    return v;
}

// One block: 32 value columns of a head.
//
// The states stay in registers, transposed: a warp has 16 columns by 32 keys as the sums of a 16 x 8 x 16 product, and
// sums are laid out as the left factors of the next, so that x, u and the states go from product to product without
// leaving their lanes; only the warps' parts of S^T k and S^T q, over 32 keys each, meet in shared memory.
// Four warps go ahead: they read rows, bring keys and queries to 16 bits of f16 (16-bit types are exact in it after a
// power of two a row, but for parts below 2^-24 of the row's length), and make A and the products P of queries and keys with
// their decays.  One inverts 1 + A by forward substitution, a column a lane, in 32 bits.
//
// Rounding: keys and queries are used as they are, and their lengths, decays and steps applied to sums in 32 bits.  S, x
// and u enter products in two f16 parts, 22 bits, and T too; the parts' products that are left out are below 2^-22 of a
// sum's terms.  What only y needs (S^T q, P u) has one part, 2^-12, where y has bf16's 2^-9, and two where it is f16.
template <typename T, int DK> __global__ void __launch_bounds__(DeltaChunk<DK>::THREADS, 1) delta_chunk_kernel(const DeltaArgs a) {
    using D = DeltaChunk<DK>;
    constexpr int C = D::C, DS = D::DS, NT = 4;            // tiles of 8 keys of a warp, and of 8 rows of a chunk
    constexpr bool FINE = std::is_same<T, __half>::value;
    constexpr int kFull = 1, kInv = 4, kFree = 7, kMeet = 10, kTeam = 12;   // barriers; the first three by slot
    constexpr int ALL = D::THREADS, STATE = 32 * D::STATE, FRONT = 32 * D::FRONT;
    extern __shared__ __align__(16) unsigned char smem[];
    const uint32_t base = tc::smem_u32(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int slice = blockIdx.x % a.slices, rest = blockIdx.x / a.slices;
    const int h = rest % a.heads, q = rest / a.heads, g = h / a.per_key, d0 = slice * kDeltaCols;
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    long long t0;
    int len;
    seq_rows(a.q, q, t0, len);
    const int chunks = (len + C - 1) / C;
    auto factors = [&](int slot) { return reinterpret_cast<float *>(smem + slot * D::SLOT + D::SC); };

    if (warp >= D::STATE && warp < D::STATE + D::FRONT) {
        // ---- ahead: rows to factors
        constexpr int VPR = DK / 8, RPP = FRONT / VPR, PASS = C / RPP;   // lanes of a row, rows at a time
        const int tid = threadIdx.x - STATE, w = warp - D::STATE, col = tid % VPR * 8, r0 = tid / VPR;
        const T *kp = static_cast<const T *>(a.kp) + (size_t)g * a.dk, *qp = static_cast<const T *>(a.qp) + (size_t)g * a.dk;
        const T *vp = static_cast<const T *>(a.vp) + (size_t)h * a.dv + d0;
        const T *dtp = static_cast<const T *>(a.dt) + h, *bp = static_cast<const T *>(a.b) + h;
        const float av = a.a[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
        uint4 kr[PASS], qr[PASS], vr;
        float dt = 0.0f, bv = 0.0f;
        auto load = [&](int c) {
#pragma unroll
            for (int p = 0; p < PASS; p++) {
                const int i = c * C + r0 + p * RPP;
                const bool live = i < len;
                const long long t = t0 + i;
                kr[p] = load_keys(kp + t * a.ld_k, col, a.dk, live, a.vec);
                qr[p] = load_keys(qp + t * a.ld_q, col, a.dk, live, a.vec);
            }
            const int i = c * C + tid / 4;
            vr = load_keys(vp + (t0 + i) * a.ld_v, tid % 4 * 8, min(a.dv - d0, kDeltaCols), i < len, a.vec_v);
            if (w == 0) {
                const bool live = c * C + lane < len;
                dt = live ? Storage<T>::to_f(dtp[(t0 + c * C + lane) * a.ld_dt]) : 0.0f;
                bv = live ? Storage<T>::to_f(bp[(t0 + c * C + lane) * a.ld_b]) : 0.0f;
            }
        };
        if (chunks) load(0);
        for (int c = 0; c < chunks; c++) {
            const int slot = c % D::SLOTS;
            if (c >= D::SLOTS) bar_sync(kFree + slot, STATE + FRONT);
            unsigned char *at = smem + slot * D::SLOT;
            float *f = factors(slot);
#pragma unroll
            for (int p = 0; p < PASS; p++)
#pragma unroll
                for (int which = 0; which < 2; which++) {
                    const uint4 raw = which ? qr[p] : kr[p];
                    const T *e = reinterpret_cast<const T *>(&raw);
                    float v[8], sq = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] = Storage<T>::to_f(e[i]), sq = fmaf(v[i], v[i], sq);
#pragma unroll
                    for (int m = 1; m < VPR; m <<= 1) sq += __shfl_xor_sync(~0u, sq, m);
                    const int row = r0 + p * RPP;
                    float down = 1.0f;
                    uint4 out = raw;
                    if (!FINE) {   // a row of length 1 to 2 times a power of two
                        const int half = ((int)(__float_as_uint(sq) >> 23) - 127) >> 1;
                        const float up = __uint_as_float((uint32_t)(127 - half) << 23);
                        down = __uint_as_float((uint32_t)(127 + half) << 23);
                        __half2 o[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) o[i] = __floats2half2_rn(v[2 * i] * up, v[2 * i + 1] * up);
                        out = *reinterpret_cast<const uint4 *>(o);
                    }
                    *reinterpret_cast<uint4 *>(at + which * D::Q + row * D::KS + col * 2) = out;
                    if (col == 0) {
                        const float norm = (a.normalize ? rsqrtf(sq + kDeltaEps) : 1.0f) * down;
                        f[(which ? kFq : kFk) * C + row] = which ? norm * a.scale : norm;
                    }
                }
            *reinterpret_cast<uint4 *>(at + D::V + tid / 4 * D::VS + tid % 4 * 16) = vr;
            if (w == 0) {
                const bool live = c * C + lane < len;
                float G = log_decay(dt + bias, av, a.softplus);
                G = !live ? 0.0f : G < -1000.0f ? -1000.0f : G;   // nothing is left below -104, and sums stay numbers
                double sum = G;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const double before = __shfl_up_sync(~0u, sum, m);
                    if (lane >= m) sum += before;
                }
                const float hi = (float)sum;
                f[kSumHi * C + lane] = hi, f[kSumLo * C + lane] = (float)(sum - hi);
                f[kBeta * C + lane] = live ? step_of(bv, a.sigmoid) : 0.0f;
            }
            bar_sync(kTeam, FRONT);
            if (c + 1 < chunks) load(c + 1);
            // products of keys (warps 0, 2) and of queries with keys (1, 3): rows 16 .. 31 (0, 1), 0 .. 15 (2, 3)
            const int m0 = w < 2 ? 16 : 0;
            const bool queries = w & 1;
            const uint32_t ka = base + slot * D::SLOT;
            float s[4][4] = {};
#pragma unroll
            for (int kk = 0; kk < DK / 16; kk++) {
                uint32_t am[4], b[2][4];
                ldsm4(am, ka + (queries ? D::Q : 0) + (m0 + lane % 16) * D::KS + kk * 32 + lane / 16 * 16);
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    if (n == 1 && m0 == 0) break;
                    ldsm4(b[n], ka + (n * 16 + lane / 16 * 8 + lane % 8) * D::KS + kk * 32 + lane / 8 % 2 * 16);
                    mma_half(s[2 * n], am, b[n][0], b[n][1]);
                    mma_half(s[2 * n + 1], am, b[n][2], b[n][3]);
                }
            }
            const int i0 = m0 + lane / 4, j0 = lane % 4 * 2;
            float hi_i[2], lo_i[2], fi[2];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const int i = i0 + 8 * r;
                hi_i[r] = f[kSumHi * C + i], lo_i[r] = f[kSumLo * C + i];
                fi[r] = queries ? f[kFq * C + i] : f[kBeta * C + i] * f[kFk * C + i];
            }
            uint32_t top[2] = {};
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int r = e / 2, i = i0 + 8 * r, j = n * 8 + j0 + e % 2;
                    const float d = (hi_i[r] - f[kSumHi * C + j]) + (lo_i[r] - f[kSumLo * C + j]);
                    const bool in = queries ? j <= i : j < i;
                    s[n][e] = in ? s[n][e] * fi[r] * f[kFk * C + j] * ex2(kLog2e * d) : 0.0f;
                    top[r] = max(top[r], magnitude(s[n][e]));
                }
            if (!queries) {
                float *A = reinterpret_cast<float *>(at + D::A);
#pragma unroll
                for (int n = 0; n < 4; n++)
#pragma unroll
                    for (int r = 0; r < 2; r++)
                        *reinterpret_cast<float2 *>(A + (i0 + 8 * r) * D::AS + n * 8 + j0) = make_float2(s[n][2 * r], s[n][2 * r + 1]);
            } else {
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    top[r] = max(top[r], __shfl_xor_sync(~0u, top[r], 1));
                    top[r] = max(top[r], __shfl_xor_sync(~0u, top[r], 2));
                    const Power p(top[r]);
                    const int i = i0 + 8 * r;
                    if (lane % 4 == 0) f[kPDown * C + i] = p.down;
#pragma unroll
                    for (int n = 0; n < 4; n++) {
                        uint32_t hi, lo;
                        split2(s[n][2 * r] * p.up, s[n][2 * r + 1] * p.up, hi, lo);
                        *reinterpret_cast<uint32_t *>(at + D::PHI + i * D::TS + n * 16 + j0 * 2) = hi;
                        if (FINE) *reinterpret_cast<uint32_t *>(at + D::PLO + i * D::TS + n * 16 + j0 * 2) = lo;
                    }
                }
            }
            if (w == 2) {   // rows' factors
                const float hi = f[kSumHi * C + lane], lo = f[kSumLo * C + lane];
                const float reach = ex2(kLog2e * hi) * (1.0f + lo), fk = f[kFk * C + lane];
                f[kBetaReach * C + lane] = f[kBeta * C + lane] * reach * fk;
                f[kQReach * C + lane] = f[kFq * C + lane] * reach;
                f[kToEnd * C + lane] = fk * ex2(kLog2e * ((f[kSumHi * C + C - 1] - hi) + (f[kSumLo * C + C - 1] - lo)));
                if (lane == C - 1) f[kTotal * C] = reach;
            }
            bar_arrive(kFull + slot, ALL);
        }
        return;
    }
    if (warp == D::STATE + D::FRONT) {
        // ---- the inverse: row i of a column is that of 1 less the rows above it, by A
        for (int c = 0; c < chunks; c++) {
            const int slot = c % D::SLOTS;
            bar_sync(kFull + slot, ALL);
            const float *A = reinterpret_cast<const float *>(smem + slot * D::SLOT + D::A);
            float t[C];
#pragma unroll
            for (int i = 0; i < C; i++) {
                float s[4] = {lane == i ? 1.0f : 0.0f};
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(A + i * D::AS + m);
                    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (m + k < i) s[k] = fmaf(-e[k], t[m + k], s[k]);
                }
                t[i] = (s[0] + s[1]) + (s[2] + s[3]);
            }
            __half *hi = reinterpret_cast<__half *>(smem + slot * D::SLOT + D::THI), *lo = reinterpret_cast<__half *>(smem + slot * D::SLOT + D::TLO);
            float mine = 0.0f;
#pragma unroll
            for (int i = 0; i < C; i++) {
                const Power p(__reduce_max_sync(~0u, magnitude(t[i])));
                const float v = t[i] * p.up;
                const __half x = __float2half_rn(v);
                hi[i * (D::TS / 2) + lane] = x;
                lo[i * (D::TS / 2) + lane] = __float2half_rn(v - __half2float(x));
                if (lane == i) mine = p.down;
            }
            factors(slot)[kTDown * C + lane] = mine;
            bar_arrive(kInv + slot, STATE + 32);
        }
        return;
    }
    // ---- the states
    const int pair = warp / DS, part = warp % DS;           // 16 columns, 32 keys
    const int rd = pair * 16 + lane / 4, k0 = part * 32;    // a lane's columns rd and rd + 8 of the block's
    const int row = a.state_in || a.state_out ? state_row(a.q, q) : -1;
    const size_t cell = ((size_t)max(row, 0) * a.heads + h) * a.dk * a.dv + d0;
    float S[NT][4];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int k = k0 + n * 8 + lane % 4 * 2 + e % 2, d = rd + e / 2 * 8;
            S[n][e] = a.state_in && row >= 0 && k < a.dk && d0 + d < a.dv ? a.state_in[cell + (size_t)k * a.dv + d] : 0.0f;
        }
    const uint32_t meet = base + D::SLOTS * D::SLOT + pair * DS * 8 * 512 + lane * 16;
    T *y = static_cast<T *>(a.y) + (size_t)h * a.dv + d0;
    for (int c = 0; c < chunks; c++) {
        const int slot = c % D::SLOTS;
        const uint32_t at = base + slot * D::SLOT;
        const float *f = factors(slot);
        uint32_t hi[NT / 2][4], lo[NT / 2][4];
        float down[2];
        as_factor(S, hi, lo, down);
        bar_sync(kFull + slot, ALL);
        float sk[NT][4] = {}, sq[NT][4] = {};
#pragma unroll
        for (int kk = 0; kk < 2; kk++)
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t b[4];
                const uint32_t p = at + (n * 8 + lane / 16 * 8 + lane % 8) * D::KS + (k0 + kk * 16 + lane / 8 % 2 * 8) * 2;
                ldsm4(b, p);
                mma_half(sk[n], hi[kk], b[0], b[1]);
                mma_half(sk[n + 1], hi[kk], b[2], b[3]);
                mma_half(sk[n], lo[kk], b[0], b[1]);
                mma_half(sk[n + 1], lo[kk], b[2], b[3]);
                ldsm4(b, p + D::Q);
                mma_half(sq[n], hi[kk], b[0], b[1]);
                mma_half(sq[n + 1], hi[kk], b[2], b[3]);
                if (FINE) {
                    mma_half(sq[n], lo[kk], b[0], b[1]);
                    mma_half(sq[n + 1], lo[kk], b[2], b[3]);
                }
            }
        const uint32_t turn = meet + (c & 1) * (2 * DS * 8 * 512);
#pragma unroll
        for (int n = 0; n < NT; n++) {
#pragma unroll
            for (int e = 0; e < 4; e++) sk[n][e] *= down[e / 2], sq[n][e] *= down[e / 2];
            tc::sts128(turn + (part * 8 + n) * 512, __float_as_uint(sk[n][0]), __float_as_uint(sk[n][1]), __float_as_uint(sk[n][2]), __float_as_uint(sk[n][3]));
            tc::sts128(turn + (part * 8 + 4 + n) * 512, __float_as_uint(sq[n][0]), __float_as_uint(sq[n][1]), __float_as_uint(sq[n][2]), __float_as_uint(sq[n][3]));
        }
        bar_sync(kMeet + pair, 32 * DS);
        // the keys' parts, in their order; then x in its place
        float x[NT][4] = {};
#pragma unroll
        for (int r = 0; r < DS; r++)
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const uint4 v = tc::lds128(turn + (r * 8 + n) * 512);
                x[n][0] += __uint_as_float(v.x), x[n][1] += __uint_as_float(v.y), x[n][2] += __uint_as_float(v.z), x[n][3] += __uint_as_float(v.w);
            }
        const T *vs = reinterpret_cast<const T *>(smem + slot * D::SLOT + D::V);
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int i = n * 8 + lane % 4 * 2 + e % 2;
                x[n][e] = fmaf(-f[kBetaReach * C + i], x[n][e], f[kBeta * C + i] * Storage<T>::to_f(vs[i * (D::VS / 2) + rd + e / 2 * 8]));
            }
        as_factor(x, hi, lo, down);
        bar_sync(kInv + slot, STATE + 32);
        float u[NT][4] = {};
#pragma unroll
        for (int n = 0; n < NT; n++) {   // rows n * 8 .. of T reach columns 0 .. n * 8 + 7
            uint32_t b[4], l[4];
            const uint32_t p = at + D::THI + (n * 8 + lane % 8) * D::TS + lane / 8 * 16;
            ldsm4(b, p);
            ldsm4(l, p + D::TLO - D::THI);
#pragma unroll
            for (int kk = 0; kk <= n / 2; kk++) {
                mma_half(u[n], hi[kk], b[2 * kk], b[2 * kk + 1]);
                mma_half(u[n], lo[kk], b[2 * kk], b[2 * kk + 1]);
                mma_half(u[n], hi[kk], l[2 * kk], l[2 * kk + 1]);
            }
        }
        float W[NT][4];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int i = n * 8 + lane % 4 * 2 + e % 2;
                u[n][e] *= down[e / 2] * f[kTDown * C + i];
                W[n][e] = u[n][e] * f[kToEnd * C + i];
            }
        // the states after the chunk
        as_factor(W, hi, lo, down);
        const float total = f[kTotal * C];
        float dS[NT][4] = {};
#pragma unroll
        for (int kk = 0; kk < 2; kk++)
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t b[4];
                ldsm4t(b, at + (kk * 16 + lane / 8 % 2 * 8 + lane % 8) * D::KS + (k0 + (n + lane / 16) * 8) * 2);
                mma_half(dS[n], hi[kk], b[0], b[1]);
                mma_half(dS[n + 1], hi[kk], b[2], b[3]);
                mma_half(dS[n], lo[kk], b[0], b[1]);
                mma_half(dS[n + 1], lo[kk], b[2], b[3]);
            }
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) S[n][e] = fmaf(dS[n][e], down[e / 2], S[n][e] * total);
        // y: this warp's share of the rows, tiles part, part + DS, ..
        as_factor(u, hi, lo, down);
#pragma unroll
        for (int n = 0; n < NT; n++) {
            if (n % DS != part) continue;
            float o[4] = {}, w[4] = {};
#pragma unroll
            for (int r = 0; r < DS; r++) {
                const uint4 v = tc::lds128(turn + (r * 8 + 4 + n) * 512);
                o[0] += __uint_as_float(v.x), o[1] += __uint_as_float(v.y), o[2] += __uint_as_float(v.z), o[3] += __uint_as_float(v.w);
            }
            uint32_t b[4], l[4];
            const uint32_t p = at + D::PHI + (n * 8 + lane % 8) * D::TS + lane / 8 * 16;
            ldsm4(b, p);
            if (FINE) ldsm4(l, p + D::PLO - D::PHI);
#pragma unroll
            for (int kk = 0; kk <= n / 2; kk++) {
                mma_half(w, hi[kk], b[2 * kk], b[2 * kk + 1]);
                if (FINE) {
                    mma_half(w, lo[kk], b[2 * kk], b[2 * kk + 1]);
                    mma_half(w, hi[kk], l[2 * kk], l[2 * kk + 1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int i = n * 8 + lane % 4 * 2 + e % 2, d = rd + e / 2 * 8;
                const float v = fmaf(w[e], down[e / 2] * f[kPDown * C + i], o[e] * f[kQReach * C + i]);
                if (c * C + i < len && d0 + d < a.dv) y[(t0 + c * C + i) * a.ld_y + d] = Storage<T>::from_f(v);
            }
        }
        if (c + D::SLOTS < chunks) bar_arrive(kFree + slot, STATE + FRONT);
    }
    if (a.state_out && row >= 0) {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int k = k0 + n * 8 + lane % 4 * 2 + e % 2, d = rd + e / 2 * 8;
                if (k < a.dk && d0 + d < a.dv) a.state_out[cell + (size_t)k * a.dv + d] = S[n][e];
            }
    }
}

}  // namespace seq
}  // namespace fcm
