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
    static constexpr int DS = 2, KW = DK / DS;        // warps that share 16 columns' states, keys of each
    static constexpr int STATE = 2 * DS, FRONT = 4;   // warps
    static constexpr int THREADS = 32 * (STATE + FRONT + 2);
    static constexpr int SLOTS = 4, AHEAD = 2;        // chunks in flight, chunks whose rows are asked for ahead
    static constexpr int KS = 2 * DK + 16;            // bytes of a row of keys: eight rows in different banks
    static constexpr int TS = 80;                     // of T's three and the rows' products' two 16-bit parts, and of values
    static constexpr int AS = 36;                     // floats of a row of A, and of T on its way
    // a slot's parts, bytes
    static constexpr int Q = C * KS, V = 2 * C * KS, TP = V + C * TS, PP = TP + 3 * C * TS, A = PP + 2 * C * TS,
                         SC = A + C * AS * 4, SLOT = SC + 8 * C * 4;
    static constexpr int XCH = 2 * 2 * DS * 8 * 512;   // sums on their way between warps: [turn][16 columns][warp][16 bytes][lane]
    static constexpr int TMP = C * AS * 4;             // T's diagonal blocks
    static constexpr int SMEM = SLOTS * SLOT + XCH + TMP;
    static_assert(AHEAD >= 2 && SLOTS > AHEAD, "a slot is waited for before its rows' factors are made");
};
// A slot's factors by row: B and B e^c / |k| (for x), e^c / |q| scale (y), e^(c_last - c) / |k| (the states).
enum { kXy = 0 /* two a row */, kQReach = 2, kToEnd, kSumHi, kSumLo, kBeta, kTotal };

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr) : "memory");
}
template <typename T> __device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
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

// The next part in bf16 of two numbers: they rounded to 8 bits, and what is left in their place, exactly.  Three parts are all
// 24 bits of a number, two are off by 2^-17 of it at most.  (Cut instead of rounded, two were off by 2^-15, always towards 0.)
__device__ __forceinline__ void part_of(float &a, float &b, uint32_t &part) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    part = *reinterpret_cast<const uint32_t *>(&h);
    a -= __uint_as_float(part << 16), b -= __uint_as_float(part & 0xFFFF0000u);
}
// N tiles of 16 x 8 sums as the left factors of the next product, in M parts of bf16.  Tiles 2 i and 2 i + 1 are 16
// inner places.
template <int M, int N> __device__ __forceinline__ void as_bf16(const float (&c)[N][4], uint32_t (&part)[3][N / 2][4]) {
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
            float a = c[i][2 * r], b = c[i][2 * r + 1];
#pragma unroll
            for (int m = 0; m < M; m++) part_of(a, b, part[m][i / 2][i % 2 * 2 + r]);
        }
}

// The same in two parts of f16, each of a lane's two rows times a power of two that its four lanes agree on;
// `down` undoes it.
template <int N>
__device__ __forceinline__ void as_half(const float (&c)[N][4], uint32_t (&part)[3][N / 2][4], float (&down)[2]) {
    uint32_t top[2];
#pragma unroll
    for (int r = 0; r < 2; r++) {
        uint32_t m[N];
#pragma unroll
        for (int i = 0; i < N; i++) m[i] = max(magnitude(c[i][2 * r]), magnitude(c[i][2 * r + 1]));
#pragma unroll
        for (int s = N / 2; s; s /= 2)
#pragma unroll
            for (int i = 0; i < s; i++) m[i] = max(m[i], m[i + s]);
        top[r] = m[0];
    }
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
            split2(c[i][2 * r] * up[r], c[i][2 * r + 1] * up[r], part[0][i / 2][i % 2 * 2 + r], part[1][i / 2][i % 2 * 2 + r]);
}

// Two 16-bit elements in 32 bits each.
template <typename T> __device__ __forceinline__ float2 two_of(uint32_t v) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    else return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Up to eight neighbouring elements of a row, zeros past its end.
template <typename T> __device__ __forceinline__ uint4 load_keys(const T *p, int n, bool live) {
    uint32_t s[8];
#pragma unroll
    for (int i = 0; i < 8; i++) s[i] = live && i < n ? reinterpret_cast<const unsigned short *>(p)[i] : 0u;
    return make_uint4(s[0] | s[1] << 16, s[2] | s[3] << 16, s[4] | s[5] << 16, s[6] | s[7] << 16);
}

// 16 bytes from global to shared memory without a register; zeros where there is no row: then nothing is read.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}

// One block: 32 value columns of a head.
//
// The states stay in registers, transposed: a warp has 16 columns by half the keys as the sums of 16 x 8 x 16 products,
// and sums are laid out as the left factors of the next, so that x, u and the states go from product to product without
// leaving their lanes; only the two halves of S^T k and S^T q meet in shared memory.  Four warps go ahead: they ask for
// rows, which enter products as they are stored, and make A and the products P of queries and keys with their decays; the
// rows' lengths are the products of keys and of queries with themselves.  One inverts 1 + A: two blocks of 16 by forward
// substitution, a column a lane, and the block below them by two products, in 32 bits.
//
// Rounding: keys and queries are used as they are, and their lengths, decays and steps applied to sums in 32 bits.  S and
// the decayed u enter products with bf16 keys in three bf16 parts, which hold all 24 bits, and with f16 keys in two f16
// parts, 22 bits, under a power of two for each column; products of second f16 parts, below 2^-22, are left out.  T and x are in three
// bf16 parts for either type (products of parts below 2^-24 are left out): T holds e^(c_i - c_j), x the rows' values beside what the
// state recalls, so that in a chunk where states grow or fall by much their numbers lie further apart than f16 reaches.
// (In two f16 parts T was infinite from 65504 on, which 32 rows of G = 0.5 pass, and had lost what it says of a state 2^14 times as large
// as the values; 503 us where these take 535.)  What only y needs has two bf16 parts, and y keeps 2^-9 or 2^-12 of itself:
// S^T q is off by 2^-17 of its terms, P u, all four products of whose parts are taken, by 2^-16.
//
// 8192 rows of 32 heads of 128 x 128, bf16, 535 us: 2.1 us a chunk, 128 blocks on as many SMs; f16 624 us.  A chunk's chain (S to
// its parts, S^T k, x, u, S again) is what it costs; with x and T in f16, 503 us in all, S^T k and q with the states' products taken
// out alone saved 103 us, the inverse 53, the rows' loads 26, the products that make A and P 18.  The tensor cores are under a half
// busy, as are the issue slots.  What was tried, us: four warps for 16 columns, 32 keys each, all factors in two f16 parts and keys
// converted in the block, 1430, two warps so 1074 (the conversions bind); products in the order of their sums, each waiting for the
// one before, 745 for 678; three slots of rows 731; S^T q's products after the meeting 503 for 499; T's parts stored one by one, as
// rows, 581 for 552.  The loops are short because the roles' code has to stay in the instruction cache together: with the inverse's
// products unrolled, and keys converted, the warps waited 2.6 cycles an instruction for their code.
//
// Four blocks make the same A, P and T, one for each 32 columns of a head.  A cluster that shares them would save some of
// the 97 us above; its blocks would wait for each other in every chunk.
template <typename T, int DK> __global__ void __launch_bounds__(DeltaChunk<DK>::THREADS, 1) delta_chunk_kernel(const DeltaArgs a) {
    using D = DeltaChunk<DK>;
    using B = __nv_bfloat16;
    constexpr int C = D::C, DS = D::DS, NS = D::KW / 8, NC = C / 8;   // tiles of 8 keys of a warp, of 8 rows of a chunk
    constexpr bool HALF = std::is_same<T, __half>::value;
    constexpr int kFull = 0, kInv = 4, kFree = 8, kMeet = 12, kTeam = 14, kRows = 15;   // barriers; the first three by slot
    constexpr int ALL = D::THREADS - 32, STATE = 32 * D::STATE, FRONT = 32 * D::FRONT;
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
    const int chunks = len / C + (len % C != 0);
    auto factors = [&](int slot) { return reinterpret_cast<float *>(smem + slot * D::SLOT + D::SC); };

    if (warp >= D::STATE && warp < D::STATE + D::FRONT) {
        // ---- ahead: rows to factors
        constexpr int VPR = DK / 8, RPP = FRONT / VPR, PASS = C / RPP;   // 16-byte pieces of a row, rows at a time
        const int tid = threadIdx.x - STATE, w = warp - D::STATE, col = tid % VPR * 8, r0 = tid / VPR;
        const T *kp = static_cast<const T *>(a.kp) + (size_t)g * a.dk, *qp = static_cast<const T *>(a.qp) + (size_t)g * a.dk;
        const T *vp = static_cast<const T *>(a.vp) + (size_t)h * a.dv + d0;
        const int vcols = min(a.dv - d0, kDeltaCols), vc = tid % 4 * 8;
        // A thread's pieces of the rows to come: where they are, and how far the next chunk's.
        const T *k_at = kp + (t0 + r0) * a.ld_k + (col < a.dk ? col : 0), *q_at = qp + (t0 + r0) * a.ld_q + (col < a.dk ? col : 0);
        const T *v_at = vp + (t0 + tid / 4) * a.ld_v + (vc < vcols ? vc : 0);
        const long long k_row = RPP * a.ld_k, q_row = RPP * a.ld_q;
        auto load = [&](int c) {
            const int slot = c % D::SLOTS;
            const uint32_t to = base + slot * D::SLOT + r0 * D::KS + col * 2, to_v = base + slot * D::SLOT + D::V + tid / 4 * D::TS + vc * 2;
            unsigned char *plain = smem + (to - base);
            const int left = len - c * C - r0;   // rows of this thread's, RPP apart
            const bool in = col < a.dk, v_live = c * C + tid / 4 < len && vc < vcols;
            const T *k = k_at, *q = q_at;
            if (a.vec && in && left >= C - r0) {   // a whole chunk's rows
#pragma unroll
                for (int p = 0; p < PASS; p++) {
                    copy16(to + p * RPP * D::KS, k, true);
                    copy16(to + D::Q + p * RPP * D::KS, q, true);
                    k += k_row, q += q_row;
                }
            } else if (a.vec) {
#pragma unroll
                for (int p = 0; p < PASS; p++) {
                    const bool live = p * RPP < left;
                    copy16(to + p * RPP * D::KS, k, live && in);
                    copy16(to + D::Q + p * RPP * D::KS, q, live && in);
                    k += k_row, q += q_row;
                }
            } else {   // element by element, all on their way before the first is stored
                uint4 ke[PASS], qe[PASS];
#pragma unroll
                for (int p = 0; p < PASS; p++) {
                    const bool live = p * RPP < left && in;
                    ke[p] = load_keys(k, a.dk - col, live), qe[p] = load_keys(q, a.dk - col, live);
                    k += k_row, q += q_row;
                }
#pragma unroll
                for (int p = 0; p < PASS; p++) {
                    *reinterpret_cast<uint4 *>(plain + p * RPP * D::KS) = ke[p];
                    *reinterpret_cast<uint4 *>(plain + D::Q + p * RPP * D::KS) = qe[p];
                }
            }
            k_at = k, q_at = q;   // PASS * RPP rows are a chunk
            if (a.vec_v) copy16(to_v, v_at, v_live);
            else *reinterpret_cast<uint4 *>(smem + (to_v - base)) = load_keys(v_at, vcols - vc, v_live);
            v_at += C * a.ld_v;
        };
#pragma unroll 1
        for (int c = -D::AHEAD; c < chunks; c++) {
            const int ahead = c + D::AHEAD;
            if (ahead < chunks) {
                if (ahead >= D::SLOTS) bar_sync(kFree + ahead % D::SLOTS, STATE + FRONT);
                load(ahead);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (c < 0) continue;
            const int slot = c % D::SLOTS;
            unsigned char *at = smem + slot * D::SLOT;
            float *f = factors(slot);
            asm volatile("cp.async.wait_group %0;" ::"n"(D::AHEAD) : "memory");
            bar_sync(kRows, FRONT + 32);
            // products of keys (warps 0, 2) and of queries with keys (1, 3): rows 0 .. 15 (0, 1: beside the two warps that
            // follow these four on the SM's schedulers), 16 .. 31 (2, 3), whose are twice as many; and of those rows with
            // themselves
            const int m0 = w < 2 ? 0 : 16;
            const bool queries = w & 1;
            const uint32_t ka = base + slot * D::SLOT, qa = ka + (queries ? D::Q : 0);
            float s[4][4] = {}, own[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < DK / 16; kk++) {
                uint32_t am[4], b[4];
                ldsm4(am, qa + (m0 + lane % 16) * D::KS + kk * 32 + lane / 16 * 16);
                const uint32_t p = (lane / 16 * 8 + lane % 8) * D::KS + kk * 32 + lane / 8 % 2 * 16;
                ldsm4(b, ka + p);
                mma16<T>(s[0], am, b[0], b[1]);
                mma16<T>(s[1], am, b[2], b[3]);
                if (m0) {
                    ldsm4(b, ka + 16 * D::KS + p);
                    mma16<T>(s[2], am, b[0], b[1]);
                    mma16<T>(s[3], am, b[2], b[3]);
                }
                ldsm4(b, qa + m0 * D::KS + p);
                mma16<T>(own[0], am, b[0], b[1]);
                mma16<T>(own[1], am, b[2], b[3]);
            }
            const int i0 = m0 + lane / 4, j0 = lane % 4 * 2;
            // the rows' own products, of row i with i: rows 0 .. 7 in tile 0, 8 .. 15 in tile 1
            float fi[2];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float mine = lane / 4 % 2 ? own[r][2 * r + 1] : own[r][2 * r];
                const float sq = __shfl_sync(~0u, mine, lane / 4 * 4 + lane / 8);
                fi[r] = a.normalize ? rsqrtf(sq + kDeltaEps) : 1.0f;
                if (lane % 4 == 0) f[(queries ? kQReach : kToEnd) * C + i0 + 8 * r] = queries ? fi[r] * a.scale : fi[r];
            }
            bar_sync(kTeam, FRONT);
            float hi_i[2], lo_i[2];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                hi_i[r] = f[kSumHi * C + i0 + 8 * r], lo_i[r] = f[kSumLo * C + i0 + 8 * r];
                fi[r] *= queries ? a.scale : f[kBeta * C + i0 + 8 * r];
            }
#pragma unroll
            for (int n = 0; n < 4; n++) {
                if (n == 2 && m0 == 0) break;   // no row before the 16th reaches these, and none is read
                const float2 hj = *reinterpret_cast<const float2 *>(f + kSumHi * C + n * 8 + j0);
                const float2 lj = *reinterpret_cast<const float2 *>(f + kSumLo * C + n * 8 + j0);
                const float2 kj = *reinterpret_cast<const float2 *>(f + kToEnd * C + n * 8 + j0);
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const int i = i0 + 8 * r, j = n * 8 + j0, last = queries ? i : i - 1;
                    const float x = s[n][2 * r] * fi[r] * kj.x * ex2((hi_i[r] - hj.x) + (lo_i[r] - lj.x));
                    const float y = s[n][2 * r + 1] * fi[r] * kj.y * ex2((hi_i[r] - hj.y) + (lo_i[r] - lj.y));
                    float2 v = make_float2(j <= last ? x : 0.0f, j + 1 <= last ? y : 0.0f);
                    if (!queries) {
                        *reinterpret_cast<float2 *>(at + D::A + (i * D::AS + j) * 4) = v;
                    } else {
                        uint32_t part;
                        part_of(v.x, v.y, part);
                        *reinterpret_cast<uint32_t *>(at + D::PP + i * D::TS + j * 2) = part;
                        part_of(v.x, v.y, part);
                        *reinterpret_cast<uint32_t *>(at + D::PP + C * D::TS + i * D::TS + j * 2) = part;
                    }
                }
            }
            bar_sync(kTeam, FRONT);   // all have read the rows' lengths, which become the rows' factors
            if (w == 1) {
                const float hi = f[kSumHi * C + lane], lo = f[kSumLo * C + lane], beta = f[kBeta * C + lane];
                const float reach = ex2(hi) * (1.0f + 0.69314718f * lo), fk = f[kToEnd * C + lane];
                *reinterpret_cast<float2 *>(f + kXy * C + 2 * lane) = make_float2(beta, beta * reach * fk);
                f[kQReach * C + lane] *= reach;
                f[kToEnd * C + lane] = fk * ex2((f[kSumHi * C + C - 1] - hi) + (f[kSumLo * C + C - 1] - lo));
                if (lane == C - 1) f[kTotal * C] = reach;
            }
            bar_arrive(kFull + slot, ALL);
        }
        return;
    }
    if (warp == D::STATE + D::FRONT + 1) {
        // ---- the rows' decays and steps, a row a lane
        const float av = a.a[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
        auto fetch = [&](const void *p, long long ld, int c) {
            const long long t = c * C + lane < len ? t0 + c * C + lane : t0;
            return Storage<T>::to_f(static_cast<const T *>(p)[t * ld + h]);
        };
        float dt_next = chunks ? fetch(a.dt, a.ld_dt, 0) : 0.0f, b_next = chunks ? fetch(a.b, a.ld_b, 0) : 0.0f;
        for (int c = 0; c < chunks; c++) {
            const int slot = c % D::SLOTS;
            const bool live = c * C + lane < len;
            const float dt = dt_next, bv = b_next;
            if (c + 1 < chunks) dt_next = fetch(a.dt, a.ld_dt, c + 1), b_next = fetch(a.b, a.ld_b, c + 1);
            float G = log_decay(dt + bias, av, a.softplus);
            G = !live ? 0.0f : G < -1000.0f ? -1000.0f : G;   // nothing is left below -104, and sums stay numbers
            double sum = G;   // differences of these sums keep a float's precision where they are small
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double before = __shfl_up_sync(~0u, sum, m);
                if (lane >= m) sum += before;
            }
            sum *= 1.4426950408889634;   // as powers of two
            const float hi = (float)sum, beta = live ? step_of(bv, a.sigmoid) : 0.0f;
            // the slot is free: the four warps have met this one for the chunk before, and waited for it earlier still
            float *f = factors(slot);
            f[kSumHi * C + lane] = hi, f[kSumLo * C + lane] = (float)(sum - hi), f[kBeta * C + lane] = beta;
            bar_sync(kRows, FRONT + 32);
        }
        return;
    }
    if (warp == D::STATE + D::FRONT) {
        // ---- the inverse.  A column of a diagonal block a lane: row i is that of 1 less the rows above it, by A.
        float *own = reinterpret_cast<float *>(smem + D::SLOTS * D::SLOT + D::XCH);
        const int j = lane % 16, half = lane / 16;
        for (int c = 0; c < chunks; c++) {
            const int slot = c % D::SLOTS;
            bar_sync(kFull + slot, ALL);
            const float *A = reinterpret_cast<const float *>(smem + slot * D::SLOT + D::A);
            const uint32_t to = base + slot * D::SLOT + D::TP;   // T's parts transposed: a lane's column lies together
            float t[16];
            const float *Ad = A + 16 * half * (D::AS + 1);
#pragma unroll
            for (int i = 0; i < 16; i++) {
                float s[2] = {j == i ? 1.0f : 0.0f};
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(Ad + i * D::AS + m);
                    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (m + k < i) s[k & 1] = fmaf(-e[k], t[m + k], s[k & 1]);
                }
                t[i] = s[0] + s[1];
                own[(16 * half + i) * D::AS + 16 * half + j] = t[i];
            }
            __syncwarp();
            // Below them -T22 A21 T11, as the transposed products T11^T A21^T and that times T22^T, whose right factors lie
            // as they are needed and whose sums are the next left factors.
            float sum[2][4];
            uint32_t left[3][1][4];
            auto times = [&](const float *from) {   // left factors by the rows of `from`
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    const float *p = from + (n * 8 + lane / 4) * D::AS + lane % 4 * 2;
                    float2 lo = *reinterpret_cast<const float2 *>(p), hi = *reinterpret_cast<const float2 *>(p + 8);
                    uint32_t b0[3], b1[3];
#pragma unroll
                    for (int m = 0; m < 3; m++) part_of(lo.x, lo.y, b0[m]), part_of(hi.x, hi.y, b1[m]);
                    float s[4] = {}, r[4] = {};   // two sums: half the chain
                    mma16<B>(r, left[2][0], b0[0], b1[0]);
                    mma16<B>(s, left[1][0], b0[0], b1[0]);
                    mma16<B>(r, left[1][0], b0[1], b1[1]);
                    mma16<B>(s, left[0][0], b0[1], b1[1]);
                    mma16<B>(r, left[0][0], b0[2], b1[2]);
                    mma16<B>(s, left[0][0], b0[0], b1[0]);
#pragma unroll
                    for (int e = 0; e < 4; e++) sum[n][e] = s[e] + r[e];
                }
            };
#pragma unroll
            for (int e = 0; e < 8; e++)   // tile e / 4 of the left factor: inner places (rows of T11) 8 (e / 4) ..
                sum[e / 4][e % 4] = own[(lane % 4 * 2 + e % 2 + e / 4 * 8) * D::AS + lane / 4 + e / 2 % 2 * 8];
            as_bf16<3>(sum, left);
            times(A + 16 * D::AS);
            as_bf16<3>(sum, left);
            times(own + 16 * (D::AS + 1));
            uint32_t p[3][8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                float x = t[2 * i], y = t[2 * i + 1];
#pragma unroll
                for (int m = 0; m < 3; m++) part_of(x, y, p[m][i]);
            }
            as_bf16<3>(sum, left);
#pragma unroll
            for (int m = 0; m < 3; m++) {
                const uint32_t at = to + m * C * D::TS, diagonal = at + lane * D::TS + half * 32;
                tc::sts128(diagonal, p[m][0], p[m][1], p[m][2], p[m][3]);
                tc::sts128(diagonal + 16, p[m][4], p[m][5], p[m][6], p[m][7]);
#pragma unroll
                for (int e = 0; e < 4; e++)   // the block below, less its sign: rows 8 (e / 2) .., columns 8 (e % 2) ..
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + (lane / 4 + e % 2 * 8) * D::TS + 32 + e / 2 * 16 + lane % 4 * 4),
                                 "r"(left[m][0][e] ^ 0x80008000u) : "memory");
            }
            __syncwarp();
            bar_arrive(kInv + slot, STATE + 32);
        }
        return;
    }
    // ---- the states
    const int pair = warp / DS, part = warp % DS;                 // 16 columns, half the keys
    const int rd = pair * 16 + lane / 4, k0 = part * D::KW;       // a lane's columns rd and rd + 8 of the block's
    const int row = a.state_in || a.state_out ? state_row(a.q, q) : -1;
    const size_t cell = ((size_t)max(row, 0) * a.heads + h) * a.dk * a.dv + d0;
    float S[NS][4];
#pragma unroll
    for (int n = 0; n < NS; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int k = k0 + n * 8 + lane % 4 * 2 + e % 2, d = rd + e / 2 * 8;
            S[n][e] = a.state_in && row >= 0 && k < a.dk && d0 + d < a.dv ? a.state_in[cell + (size_t)k * a.dv + d] : 0.0f;
        }
    const uint32_t meet = base + D::SLOTS * D::SLOT + pair * DS * 8 * 512 + lane * 16;
    T *y_at = static_cast<T *>(a.y) + (size_t)h * a.dv + d0 + rd + (t0 + part * 8 + lane % 4 * 2) * a.ld_y;   // a lane's first row
    const bool in0 = d0 + rd < a.dv, in1 = d0 + rd + 8 < a.dv;
    for (int c = 0; c < chunks; c++) {
        const int slot = c % D::SLOTS;
        const uint32_t at = base + slot * D::SLOT;
        const float *f = factors(slot);
        float sk[NC][4] = {}, sq[NC][4] = {};
        {
            uint32_t sp[3][NS / 2][4];
            float down[2] = {1.0f, 1.0f};
            if constexpr (HALF) as_half(S, sp, down);
            else as_bf16<3>(S, sp);
            bar_sync(kFull + slot, ALL);
            // Every sum of products goes round its tiles, so that one product does not wait for the one before: a product's
            // sum is there after 21 cycles, and the next may begin after 8.
            const uint32_t keys = at + (lane / 16 * 8 + lane % 8) * D::KS + (k0 + lane / 8 % 2 * 8) * 2;
#pragma unroll
            for (int kk = 0; kk < NS / 2; kk++) {
                uint32_t b[2][4];
#pragma unroll
                for (int i = 0; i < 2; i++) ldsm4(b[i], keys + i * 16 * D::KS + kk * 32);
#pragma unroll
                for (int m = 0; m < (HALF ? 2 : 3); m++)
#pragma unroll
                    for (int n = 0; n < NC; n++) mma16<T>(sk[n], sp[m][kk], b[n / 2][n % 2 * 2], b[n / 2][n % 2 * 2 + 1]);
#pragma unroll
                for (int i = 0; i < 2; i++) ldsm4(b[i], keys + D::Q + i * 16 * D::KS + kk * 32);
#pragma unroll
                for (int m = 0; m < 2; m++)
#pragma unroll
                    for (int n = 0; n < NC; n++) mma16<T>(sq[n], sp[m][kk], b[n / 2][n % 2 * 2], b[n / 2][n % 2 * 2 + 1]);
            }
            if (HALF)
#pragma unroll
                for (int n = 0; n < NC; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) sk[n][e] *= down[e / 2], sq[n][e] *= down[e / 2];
        }
        // the halves meet: all of S^T k, and of S^T q the tiles that the other warp finishes (this one: part, part + 2)
        const uint32_t turn = meet + (c & 1) * (2 * DS * 8 * 512);
        const uint32_t mine = turn + part * 8 * 512, other = turn + (part ^ 1) * 8 * 512;
        auto give = [&](int i, const float (&v)[4]) {
            tc::sts128(mine + i * 512, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        };
        auto take = [&](int i, float (&v)[4]) {   // the sum of two is the same in either order
            const uint4 o = tc::lds128(other + i * 512);
            v[0] += __uint_as_float(o.x), v[1] += __uint_as_float(o.y), v[2] += __uint_as_float(o.z), v[3] += __uint_as_float(o.w);
        };
        float yq[2][4];
#pragma unroll
        for (int n = 0; n < NC; n++) give(n, sk[n]);
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                yq[i][e] = part ? sq[2 * i + 1][e] : sq[2 * i][e];
                sq[i][e] = part ? sq[2 * i][e] : sq[2 * i + 1][e];
            }
        give(4, sq[0]), give(5, sq[1]);
        bar_sync(kMeet + pair, 32 * DS);
#pragma unroll
        for (int n = 0; n < NC; n++) take(n, sk[n]);
        take(4, yq[0]), take(5, yq[1]);
        // x in the place of S^T k
        float u[NC][4] = {};
        {
            uint32_t xp[3][NC / 2][4];
            uint32_t v[2][4];   // values of eight columns and all rows, transposed: a lane's column, two rows a register
#pragma unroll
            for (int i = 0; i < 2; i++) ldsm4t(v[i], at + D::V + lane * D::TS + (pair * 16 + i * 8) * 2);
#pragma unroll
            for (int n = 0; n < NC; n++) {
                const float4 w = *reinterpret_cast<const float4 *>(f + kXy * C + 2 * (n * 8 + lane % 4 * 2));   // B, .. of two rows
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float2 x = two_of<T>(v[i][n]);
                    sk[n][2 * i] = fmaf(-w.y, sk[n][2 * i], w.x * x.x);
                    sk[n][2 * i + 1] = fmaf(-w.w, sk[n][2 * i + 1], w.z * x.y);
                }
            }
            as_bf16<3>(sk, xp);
            bar_sync(kInv + slot, STATE + 32);
#pragma unroll
            for (int m = 2; m >= 0; m--) {   // rows n * 8 .. of T reach columns 0 .. n * 8 + 7
                uint32_t b[NC][4];
#pragma unroll
                for (int n = 0; n < NC; n++) ldsm4t(b[n], at + D::TP + m * C * D::TS + lane * D::TS + n * 16);
#pragma unroll
                for (int l = 2 - m; l >= 0; l--)
#pragma unroll
                    for (int kk = 0; kk < NC / 2; kk++)
#pragma unroll
                        for (int n = 2 * kk; n < NC; n++) mma16<B>(u[n], xp[l][kk], b[n][2 * kk], b[n][2 * kk + 1]);
            }
        }
        // the states after the chunk
        const float total = f[kTotal * C];
        {
            uint32_t wp[3][NC / 2][4];
            float W[NC][4], down[2];
#pragma unroll
            for (int n = 0; n < NC; n++) {
                const float2 w = *reinterpret_cast<const float2 *>(f + kToEnd * C + n * 8 + lane % 4 * 2);
#pragma unroll
                for (int e = 0; e < 4; e++) W[n][e] = u[n][e] * (e % 2 ? w.y : w.x);
            }
            if constexpr (HALF) as_half(W, wp, down);
            else as_bf16<3>(W, wp);
            float add[NS][4];
#pragma unroll
            for (int n = 0; n < NS; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    S[n][e] *= total;
                    add[n][e] = HALF ? 0.0f : S[n][e];
                }
#pragma unroll
            for (int kk = 0; kk < NC / 2; kk++) {
                uint32_t b[NS / 2][4];
#pragma unroll
                for (int i = 0; i < NS / 2; i++)
                    ldsm4t(b[i], at + (kk * 16 + lane / 8 % 2 * 8 + lane % 8) * D::KS + (k0 + (2 * i + lane / 16) * 8) * 2);
#pragma unroll
                for (int m = 0; m < (HALF ? 2 : 3); m++)
#pragma unroll
                    for (int n = 0; n < NS; n++) mma16<T>(add[n], wp[m][kk], b[n / 2][n % 2 * 2], b[n / 2][n % 2 * 2 + 1]);
            }
#pragma unroll
            for (int n = 0; n < NS; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) S[n][e] = HALF ? fmaf(add[n][e], down[e / 2], S[n][e]) : add[n][e];
        }
        // y of this warp's tiles of rows
        {
            uint32_t up[3][NC / 2][4];
            as_bf16<2>(u, up);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int n = 2 * i + part;
                float w[4] = {};
                uint32_t b[2][4];
                const uint32_t p = at + D::PP + (n * 8 + lane % 8) * D::TS + lane / 8 * 16;
                ldsm4(b[0], p);
                ldsm4(b[1], p + C * D::TS);
#pragma unroll
                for (int kk = 0; kk <= i; kk++) {
#pragma unroll
                    for (int m = 3; m >= 0; m--) mma16<B>(w, up[m % 2][kk], b[m / 2][2 * kk], b[m / 2][2 * kk + 1]);
                }
                const int r = n * 8 + lane % 4 * 2, live = len - c * C - r;   // rows r and r + 1
                const float2 reach = *reinterpret_cast<const float2 *>(f + kQReach * C + r);
                T *to = y_at + i * 16 * a.ld_y;
                if (live > 0 && in0) to[0] = Storage<T>::from_f(fmaf(yq[i][0], reach.x, w[0]));
                if (live > 0 && in1) to[8] = Storage<T>::from_f(fmaf(yq[i][2], reach.x, w[2]));
                to += a.ld_y;
                if (live > 1 && in0) to[0] = Storage<T>::from_f(fmaf(yq[i][1], reach.y, w[1]));
                if (live > 1 && in1) to[8] = Storage<T>::from_f(fmaf(yq[i][3], reach.y, w[3]));
            }
        }
        y_at += C * a.ld_y;
        if (c + D::SLOTS < chunks) bar_arrive(kFree + slot, STATE + FRONT);
    }
    if (a.state_out && row >= 0) {
#pragma unroll
        for (int n = 0; n < NS; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int k = k0 + n * 8 + lane % 4 * 2 + e % 2, d = rd + e / 2 * 8;
                if (k < a.dk && d0 + d < a.dv) a.state_out[cell + (size_t)k * a.dv + d] = S[n][e];
            }
    }
}

}  // namespace seq
}  // namespace fcm
