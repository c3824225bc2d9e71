// seq_scan.cuh -- the selective scan's prompt kernel.
//
//     h[d,n] = exp(D * a[d,n]) * h[d,n] + D * x[t,d] * bm[t,g,n],   D = softplus(dt[t,d] + dt_bias[d])
//     y[t,d] = (sum_n cm[t,g,n] * h[d,n] + skip[d] * x[t,d]) * silu(z[t,d])
#pragma once


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
    int cpg;        // channels per group
    int blocks;     // channel blocks per group
    int vec16;      // every block's row of x, dt and z starts on 16 bytes
    int vec16n;     // every row of bm and cm starts on 16 bytes
    int vec2;       // every block's row of y starts on two elements
};

constexpr int kMaxState = 128;

// ------------------------------------------------------------------ arithmetic
// Two 32-bit floats in one register pair: the packed forms halve the instructions issued (the
// multiply-add pipe's rate is the same).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// max(v, 0) + log(1 + e^-|v|) of two values.  log(1 + t) / t on [0, 1] is the polynomial of degree
// 9 whose largest relative error is least (Remez exchange in 64 bits): 5e-9, with 32-bit
// arithmetic 2.5 * 2^-24.  So the relative precision stays where v is far below 0.
__device__ __forceinline__ void softplus2(float &a, float &b) {
    constexpr float c[10] = {-0.0032440251670777798f, 0.01985146291553974f, -0.05695953592658043f,
                             0.10603655129671097f, -0.15305592119693756f, 0.1967593878507614f,
                             -0.24954134225845337f, 0.3332996368408203f, -0.4999990165233612f, 1.0f};
    const f32x2 t = pack2(ex2(-kLog2e * fabsf(a)), ex2(-kLog2e * fabsf(b)));
    f32x2 p = pack2(c[0], c[0]);
#pragma unroll
    for (int i = 1; i < 10; i++) p = fma2(p, t, pack2(c[i], c[i]));
    unpack2(fma2(p, t, pack2(fmaxf(a, 0.0f), fmaxf(b, 0.0f))), a, b);
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t local, int rank) {
    uint32_t addr;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Two states carried through a part's rows, whose decays multiply to 2^t, plus what the part makes from
// zero; third: t / 3.  t may be far outside a float's exponents where h, or the result, is not, and a
// factor of 0 or infinity would make NaN of an infinite h or of one of 0.  2^(t / 3), cut to normal
// numbers and multiplied three times, is neither, and still takes any h that is not 0 past either end.
__device__ __forceinline__ f32x2 carry2(f32x2 h, f32x2 third, f32x2 from_zero) {
    float lo, hi;
    unpack2(third, lo, hi);
    const f32x2 f = pack2(ex2(fminf(fmaxf(lo, -126.0f), 126.0f)), ex2(fminf(fmaxf(hi, -126.0f), 126.0f)));
    return fma2(mul2(mul2(h, f), f), f, from_zero);
}

// ------------------------------------------------------------------ copies to shared memory
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile's rows lie 16 bytes further apart than their length, which keeps lanes that read different
// rows on different banks.  16-byte aligned rows are copied in 16-byte pieces; others in the
// aligned pieces that hold their bytes, each row at the offset that its address has within a
// piece (an allocation starts on a piece, so that the bytes before the row are mapped; of the last
// piece no more than the row is read).
// What lies past a tile's rows or a row's elements is not used.
constexpr int row_pitch(int rb) { return (rb < 16 ? 16 : rb) + 16; }
// A barrier of the four warps that do not scan.
__device__ __forceinline__ void helpers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Two neighbouring elements in shared memory, widened; whole: their address is a multiple of both.
template <typename T> __device__ __forceinline__ void get_pair(const unsigned char *p, bool whole, float &a, float &b) {
    if (whole) {
        if constexpr (sizeof(T) == 4) {
            const float2 v = *reinterpret_cast<const float2 *>(p);
            a = v.x, b = v.y;
        } else {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
            if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
                a = f.x, b = f.y;
            } else {
                a = __uint_as_float(v << 16), b = __uint_as_float(v & 0xFFFF0000u);
            }
        }
    } else {
        a = Storage<T>::to_f(*reinterpret_cast<const T *>(p));
        b = Storage<T>::to_f(*reinterpret_cast<const T *>(p + sizeof(T)));
    }
}
template <typename T> __device__ __forceinline__ void store_pair(T *p, float a, float b, int have, bool vec2) {
    if (vec2 && have >= 2) {
        const float v[2] = {a, b};
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float2 *>(p) = make_float2(a, b);
        } else if constexpr (std::is_same<T, __half>::value) {
            *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(v[0], v[1]);
        } else {
            *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
        }
    } else {
        if (have >= 1) p[0] = Storage<T>::from_f(a);
        if (have >= 2) p[1] = Storage<T>::from_f(b);
    }
}

// ------------------------------------------------------------------ the kernel
// SPT states per thread, LPC lanes per channel (SPT * LPC >= n).  PAD: 0, n is their product; 1, a
// lane's states all exist or none does; 2, neither.  Four warps scan:
// a warp holds 32 / LPC channels, lane = part * channels + channel, so that the lanes that read
// one part of B and C are neighbours and the read is a broadcast.  Four more warps do what is
// per channel and token: they load, make the steps D and D * x and widen B and C for the tile
// behind, and sum the parts' products, gate and store the tile before.
//
// Bound by shared memory (its pipe is 76 % busy: steps, widened B and C, partial sums) and by the latencies
// of the one scanning warp and the one helping warp that each scheduler has (two of each, where two blocks share
// an SM; issue is at 49 %): 8192 x 4096, 16 states, bf16: 245 us, 58 cycles a row, where its exponentials
// take 56 us at the SM's 32 a clock and its 269 MB 40; the scanning warps by themselves would take 155.
// 4 x 2048 x 4096, two blocks an SM, 176; rows off 16 bytes, 8192 x 4095, 344. What gave that: warps that do
// nothing but scan 447 -> 282, their rows in three stages and the helpers' two tiles side by side 282 -> 249.
// What gave nothing: more or split teams of helpers, two states a lane (403 against 282) and single in place of
// packed products (288).
constexpr int scan_rows(int ch, int np) { return 1024 / ch < 32 ? 1024 / ch : np >= 64 ? 16 : 32; }
template <typename T, int SPT, int LPC> struct ScanShape {
    static constexpr int NS = 128, NT = 256;     // scanning threads, threads
    static constexpr int CHW = 32 / LPC;         // channels per warp
    static constexpr int CH = 4 * CHW;           // channels per block
    static constexpr int NP = SPT * LPC;         // states, padded
    static constexpr int TT = scan_rows(CH, NP);   // rows per tile
    static constexpr int NST = 5;                // tiles on chip: one of them finished, one scanned,
                                                 // one prepared, two on their way
    static constexpr int RBX = CH * (int)sizeof(T), RBN = NP * (int)sizeof(T);
    static constexpr int X_BYTES = TT * row_pitch(RBX), N_BYTES = TT * row_pitch(RBN);
    static constexpr int STAGE = 3 * X_BYTES + 2 * N_BYTES;   // x, dt, z, B, C as stored
    static constexpr int DU = TT * CH * 8;       // D and D * x of a tile
    static constexpr int BC = TT * 2 * NP * 4;   // B and C of a tile, widened
    static constexpr int OUT = TT * CH * LPC * 4;
    static constexpr int JOIN = NS * (SPT + 1) * 4;   // what the parts of a sequence hand on
    static constexpr int SMEM = NST * STAGE + 2 * (DU + BC + OUT);   // and JOIN where sequences are split
};

template <typename T, int SPT, int LPC, int PAD, bool SPLIT>
__global__ void __launch_bounds__(256, 2) scan_kernel(const ScanArgs a) {
    typedef ScanShape<T, SPT, LPC> S;
    constexpr int TT = S::TT, CH = S::CH, CHW = S::CHW, NP = S::NP;
    extern __shared__ __align__(16) unsigned char smem[];

    tc::pdl_wait();
    tc::pdl_launch_dependents();

    const int parts = SPLIT ? (int)cluster_size() : 1;
    const int rank = SPLIT ? (int)(blockIdx.x % parts) : 0;
    int id = SPLIT ? (int)(blockIdx.x / parts) : (int)blockIdx.x;
    const int block = id % a.blocks;
    id /= a.blocks;
    const int g = id % a.groups, q = id / a.groups;
    long long start;
    int len;
    seq_rows(a.q, q, start, len);
    const int row = a.state_in || a.state_out ? state_row(a.q, q) : -1;
    const int valid = min(CH, a.cpg - block * CH);              // the block's channels
    const long long c0 = (long long)g * a.cpg + block * CH;     // the first one
    // this part's rows
    const unsigned all = (unsigned)len;   // sums with it may pass 2^31
    const unsigned per = SPLIT ? ((all + parts - 1) / parts + TT - 1) / TT * TT : all;
    const int t0 = SPLIT ? (int)min(all, rank * per) : 0, t1 = SPLIT ? (int)min(all, t0 + per) : len;
    const int tiles = (int)(((unsigned)(t1 - t0) + TT - 1) / TT);
    auto at_du = [&](int k) { return reinterpret_cast<float2 *>(smem + S::NST * S::STAGE + (k & 1) * S::DU); };
    auto at_bc = [&](int k) { return reinterpret_cast<float *>(smem + S::NST * S::STAGE + 2 * S::DU + (k & 1) * S::BC); };
    auto at_out = [&](int k) { return reinterpret_cast<float *>(smem + S::NST * S::STAGE + 2 * (S::DU + S::BC) + (k & 1) * S::OUT); };

    if (threadIdx.x < S::NS) {
        // ---------------------------------------------------------------- scanning warps
        const int tid = threadIdx.x, lane = tid & 31, part = lane / CHW, n0 = part * SPT;
        const int cb = (tid >> 5) * CHW + lane % CHW;           // channel in the block
        const bool live = cb < valid;
        const size_t at = (size_t)(c0 + (live ? cb : 0)) * a.n + n0;
        f32x2 av[SPT / 2], h0[SPT / 2], h[SPT / 2];   // decays (base 2), states before, states
        {
            float v[SPT], w[SPT];
#pragma unroll
            for (int i = 0; i < SPT; i++) {
                const bool in = live && (PAD == 0 || n0 + i < a.n);
                v[i] = in ? a.a[at + i] * kLog2e : 0.0f;
                w[i] = in && row >= 0 && a.state_in ? a.state_in[(size_t)row * a.c * a.n + at + i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < SPT / 2; i++) av[i] = pack2(v[2 * i], v[2 * i + 1]), h0[i] = pack2(w[2 * i], w[2 * i + 1]);
        }
        float sum_d = 0.0f;
        // the tiles, with or without the products with C
        auto scan = [&](auto out_tag) {
            constexpr bool OUT = decltype(out_tag)::value;
            __syncthreads();
            for (int k = 0; k < tiles; k++) {
                float tile_d = 0.0f;   // the tile's steps by themselves: their sum's error is a short one's
                const float2 *du = at_du(k) + cb;
                const float *bc = at_bc(k) + n0;
                float *out = at_out(k) + cb * LPC + part;
                auto step = [&](int r) {
                    const float2 s = du[r * CH];
                    const f32x2 u2 = pack2(s.y, s.y), d2 = pack2(s.x, s.x);
                    if (SPLIT && !OUT) tile_d += s.x;
                    f32x2 acc0 = 0, acc1 = 0;
#pragma unroll
                    for (int j = 0; j < SPT / 2; j += 2) {
                        const ulonglong2 b2 = *reinterpret_cast<const ulonglong2 *>(bc + r * 2 * NP + 2 * j);
                        float e0, e1, e2, e3;
                        unpack2(mul2(d2, av[j]), e0, e1);
                        unpack2(mul2(d2, av[j + 1]), e2, e3);
                        h[j] = fma2(pack2(ex2(e0), ex2(e1)), h[j], mul2(u2, b2.x));
                        h[j + 1] = fma2(pack2(ex2(e2), ex2(e3)), h[j + 1], mul2(u2, b2.y));
                        if (OUT) {
                            const ulonglong2 c2 = *reinterpret_cast<const ulonglong2 *>(bc + r * 2 * NP + NP + 2 * j);
                            f32x2 s0 = h[j], s1 = h[j + 1];
                            if (PAD == 2) {   // a padding state's 0 * infinity stays out of the sum
                                float p0, p1, p2, p3;
                                unpack2(s0, p0, p1);
                                unpack2(s1, p2, p3);
                                const int n = n0 + 2 * j;
                                s0 = pack2(n < a.n ? p0 : 0.0f, n + 1 < a.n ? p1 : 0.0f);
                                s1 = pack2(n + 2 < a.n ? p2 : 0.0f, n + 3 < a.n ? p3 : 0.0f);
                            }
                            acc0 = j == 0 ? mul2(s0, c2.x) : fma2(s0, c2.x, acc0);
                            acc1 = j == 0 ? mul2(s1, c2.y) : fma2(s1, c2.y, acc1);
                        }
                    }
                    float lo, hi;
                    unpack2(add2(acc0, acc1), lo, hi);
                    return PAD == 1 && n0 >= a.n ? 0.0f : lo + hi;
                };
                const int rows = min(TT, t1 - t0 - k * TT);
                if (rows == TT) {
                    // Three stages of R rows each: loads, exponentials, and the recurrence; a batch's
                    // sums are stored behind the next one's loads.
                    constexpr int R = 16 / SPT, NB = TT / R, H = SPT / 2;
                    static_assert(R * SPT == 16 && NB * R == TT, "batches fill the tile");
                    static_assert(NB >= 2, "two batches are loaded before the first is used");
                    static_assert(SPT % 4 == 0, "a lane's part of B and C is whole 16-byte loads");
                    struct In {
                        float2 s[R];
                        ulonglong2 b[R][H / 2], c[R][H / 2];
                    };
                    struct Mid {
                        f32x2 e[R][H], u[R][H];
                    };
                    auto load = [&](In &x, int r0) {
#pragma unroll
                        for (int i = 0; i < R; i++) {
                            x.s[i] = du[(r0 + i) * CH];
#pragma unroll
                            for (int j = 0; j < H / 2; j++) {
                                x.b[i][j] = *reinterpret_cast<const ulonglong2 *>(bc + (r0 + i) * 2 * NP + 4 * j);
                                if (OUT) x.c[i][j] = *reinterpret_cast<const ulonglong2 *>(bc + (r0 + i) * 2 * NP + NP + 4 * j);
                            }
                        }
                    };
                    auto factors = [&](Mid &m, const In &x) {
#pragma unroll
                        for (int i = 0; i < R; i++) {
                            const f32x2 u2 = pack2(x.s[i].y, x.s[i].y), d2 = pack2(x.s[i].x, x.s[i].x);
                            if (SPLIT && !OUT) tile_d += x.s[i].x;
#pragma unroll
                            for (int j = 0; j < H; j++) {
                                float e0, e1;
                                unpack2(mul2(d2, av[j]), e0, e1);
                                m.e[i][j] = pack2(ex2(e0), ex2(e1));
                                m.u[i][j] = mul2(u2, j & 1 ? x.b[i][j / 2].y : x.b[i][j / 2].x);
                            }
                        }
                    };
                    auto advance = [&](const Mid &m, const In &x, float (&sums)[R]) {
#pragma unroll
                        for (int i = 0; i < R; i++) {
                            f32x2 acc[2] = {0, 0};
#pragma unroll
                            for (int j = 0; j < H; j++) {
                                h[j] = fma2(m.e[i][j], h[j], m.u[i][j]);
                                if (OUT) {
                                    f32x2 v = h[j];
                                    if (PAD == 2) {
                                        float p0, p1;
                                        unpack2(v, p0, p1);
                                        v = pack2(n0 + 2 * j < a.n ? p0 : 0.0f, n0 + 2 * j + 1 < a.n ? p1 : 0.0f);
                                    }
                                    const f32x2 c = j & 1 ? x.c[i][j / 2].y : x.c[i][j / 2].x;
                                    acc[j & 1] = j < 2 ? mul2(v, c) : fma2(v, c, acc[j & 1]);
                                }
                            }
                            float lo, hi;
                            unpack2(add2(acc[0], acc[1]), lo, hi);
                            sums[i] = PAD == 1 && n0 >= a.n ? 0.0f : lo + hi;
                        }
                    };
                    In x[3];
                    Mid m[2];
                    float sums[R];
                    load(x[0], 0);
                    load(x[1], R);
                    factors(m[0], x[0]);
#pragma unroll
                    for (int k0 = 0; k0 < NB; k0++) {
                        if (k0 + 2 < NB) load(x[(k0 + 2) % 3], (k0 + 2) * R);
                        if (OUT && k0 > 0)
#pragma unroll
                            for (int i = 0; i < R; i++) out[((k0 - 1) * R + i) * CH * LPC] = sums[i];
                        if (k0 + 1 < NB) factors(m[(k0 + 1) & 1], x[(k0 + 1) % 3]);
                        advance(m[k0 & 1], x[k0 % 3], sums);
                    }
                    if (OUT)
#pragma unroll
                        for (int i = 0; i < R; i++) out[((NB - 1) * R + i) * CH * LPC] = sums[i];
                } else {
#pragma unroll 1
                    for (int r = 0; r < rows; r++) {
                        const float sum = step(r);
                        if (OUT) out[r * CH * LPC] = sum;
                    }
                }
                if (SPLIT && !OUT) sum_d += tile_d;
                __syncthreads();
            }
        };
        if constexpr (SPLIT) {
            // Each part but the last runs from zero; a part's start is the state before the first
            // one, carried through the parts between: h = exp(a * sum of their steps) * h + theirs (carry2).
            float *join = reinterpret_cast<float *>(smem + S::SMEM);
#pragma unroll
            for (int i = 0; i < SPT / 2; i++) h[i] = 0;
            if (rank + 1 < parts) scan(std::false_type{});
#pragma unroll
            for (int i = 0; i < SPT / 2; i++) {
                float lo, hi;
                unpack2(h[i], lo, hi);
                join[2 * i * S::NS + tid] = lo;
                join[(2 * i + 1) * S::NS + tid] = hi;
            }
            join[SPT * S::NS + tid] = sum_d;
            cluster_sync();
            const uint32_t join_at = tc::smem_u32(join);
            for (int p = 0; p < rank; p++) {
                const float s = ld_cluster(join_at + (SPT * S::NS + tid) * 4, p) * (1.0f / 3.0f);
#pragma unroll
                for (int i = 0; i < SPT / 2; i++)
                    h0[i] = carry2(h0[i], mul2(pack2(s, s), av[i]),
                                   pack2(ld_cluster(join_at + (2 * i * S::NS + tid) * 4, p),
                                         ld_cluster(join_at + ((2 * i + 1) * S::NS + tid) * 4, p)));
            }
        }
#pragma unroll
        for (int i = 0; i < SPT / 2; i++) h[i] = h0[i];
        scan(std::true_type{});
        if (rank == parts - 1 && row >= 0 && a.state_out && live) {
            float *to = a.state_out + (size_t)row * a.c * a.n + at;
#pragma unroll
            for (int i = 0; i < SPT; i++) {
                float lo, hi;
                unpack2(h[i / 2], lo, hi);
                if (PAD == 0 || n0 + i < a.n) to[i] = i & 1 ? hi : lo;
            }
        }
    } else {
        // ---------------------------------------------------------------- the others
        const int tid = threadIdx.x - S::NS;
        auto help = [&](auto vec_tag, auto vecn_tag) {
            constexpr bool vec16 = decltype(vec_tag)::value, vec16n = decltype(vecn_tag)::value;
            constexpr int E = (int)sizeof(T), NST = S::NST, PITCHX = row_pitch(S::RBX), PITCHN = row_pitch(S::RBN);
            const uint32_t sm = tc::smem_u32(smem);
            const long long bx = a.ld_x * E, bdt = a.ld_dt * E, bz = a.ld_z * E, bb = a.ld_b * E, bc = a.ld_c * E;
            const long long first = start + t0;
            const char *px = static_cast<const char *>(a.x) + first * bx + c0 * E;
            const char *pdt = static_cast<const char *>(a.dt) + first * bdt + c0 * E;
            const char *pz = static_cast<const char *>(a.z) + (a.z ? first * bz + c0 * E : 0);
            const char *pb = static_cast<const char *>(a.bm) + first * bb + (long long)g * a.n * E;
            const char *pc = static_cast<const char *>(a.cm) + first * bc + (long long)g * a.n * E;

            // ---- copies: a tile's rows, asynchronously, two tiles ahead of their use
            constexpr int NPX = (S::RBX < 16 ? 1 : S::RBX / 16) + !vec16;   // pieces of a row
            constexpr int NPN = (S::RBN < 16 ? 1 : S::RBN / 16) + !vec16n;
            constexpr int RX = 128 / NPX < TT ? 128 / NPX : TT, RN = 128 / NPN < TT ? 128 / NPN : TT; // rows at once
            const int rx = tid / NPX, qx = tid % NPX * 16, rn = tid / NPN, qn = tid % NPN * 16;
            const int nx = rx < TT ? max(0, min(16, valid * E - qx)) : 0, nn = rn < TT ? max(0, min(16, a.n * E - qn)) : 0;
            auto copy = [&](auto rows_tag, auto pitch_tag, uint32_t to, const char *from, long long stride, int r, int n, int rows) {
                constexpr int R = decltype(rows_tag)::value, PITCH = decltype(pitch_tag)::value;
                if (n > 0) {
#pragma unroll
                    for (int i = 0; i < TT; i += R)
                        if (r + i < rows) cp_async16(to + i * PITCH, from + i * stride, n);
                }
            };
            auto copy_any = [&](auto rows_tag, auto pitch_tag, uint32_t to, const char *from, long long stride, int r, int q, int n, int rows) {
                constexpr int R = decltype(rows_tag)::value, PITCH = decltype(pitch_tag)::value;
                if (r >= R) return;   // the last threads, where the pieces do not divide them
#pragma unroll
                for (int i = 0; i < TT; i += R) {
                    const char *p = from + i * stride;
                    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15), m = min(16, n + off - q);
                    if ((TT % R == 0 || r + i < TT) && r + i < rows && m > 0) cp_async16(to + i * PITCH, p - off, m);
                }
            };
            typedef std::integral_constant<int, RX> RowsX;
            typedef std::integral_constant<int, RN> RowsN;
            typedef std::integral_constant<int, PITCHX> PitchX;
            typedef std::integral_constant<int, PITCHN> PitchN;
            const char *sx = px + rx * bx + qx, *sdt = pdt + rx * bdt + qx, *sz = pz + rx * bz + qx;
            const char *sb = pb + rn * bb + qn, *sc = pc + rn * bc + qn;
            auto stage = [&](int k, bool with_out) {
                if (k < tiles) {
                    const uint32_t at = sm + (k % NST) * S::STAGE;
                    const int rows = t1 - t0 - k * TT;
                    const uint32_t ax = at + rx * PITCHX + qx, an = at + 3 * S::X_BYTES + rn * PITCHN + qn;
                    auto copy_x = [&](uint32_t to, const char *from, long long stride) {
                        if constexpr (vec16) copy(RowsX{}, PitchX{}, to, from, stride, rx, nx, rows);
                        else copy_any(RowsX{}, PitchX{}, to, from, stride, rx, qx, valid * E, rows);
                    };
                    auto copy_n = [&](uint32_t to, const char *from, long long stride) {
                        if constexpr (vec16n) copy(RowsN{}, PitchN{}, to, from, stride, rn, nn, rows);
                        else copy_any(RowsN{}, PitchN{}, to, from, stride, rn, qn, a.n * E, rows);
                    };
                    copy_x(ax, sx, bx);
                    copy_x(ax + S::X_BYTES, sdt, bdt);
                    copy_n(an, sb, bb);
                    if (with_out) {
                        if (a.z) copy_x(ax + 2 * S::X_BYTES, sz, bz);
                        copy_n(an + S::N_BYTES, sc, bc);
                    }
                    sx += TT * bx, sdt += TT * bdt, sz += TT * bz, sb += TT * bb, sc += TT * bc;
                }
                cp_commit();
            };

            // ---- channel pairs of a tile, and quads of states
            constexpr int PR = CH / 2, RS = 128 / PR < TT ? 128 / PR : TT, IT = TT / RS;
            constexpr int QR = NP / 4, QS = 128 / QR < TT ? 128 / QR : TT, QT = TT / QS;
            const int ch = tid % PR * 2, r0 = tid / PR, have = r0 < RS ? valid - ch : 0;
            const int n4 = tid % QR * 4, rq = tid / QR;
            float bias[2] = {0.0f, 0.0f}, skip[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 2; i++)
                if (have > i) {
                    if (a.dt_bias) bias[i] = a.dt_bias[c0 + ch + i];
                    if (a.skip) skip[i] = a.skip[c0 + ch + i];
                }
            T *py = static_cast<T *>(a.y) + (first + r0) * a.ld_y + c0 + ch;
            // where row r of a tile starts within its place: the copies keep the address's rest
            auto rest = [&](const char *p, long long stride, uint32_t r) {
                return ((uint32_t)reinterpret_cast<uintptr_t>(p) + r * (uint32_t)stride) & 15;
            };
            // PREP: the steps and widened B and C of tile k + 1; OUT: the outputs of tile k - 1.  Everything is
            // read before anything is written, so that the two tiles' chains run side by side; where there
            // is no such tile, what lies in its place is worked on and not used.
            auto serve_tile = [&](auto prep_tag, auto c_tag, auto out_tag, auto gate_tag, int k) {
                constexpr bool PREP = decltype(prep_tag)::value, WITH_C = decltype(c_tag)::value;
                constexpr bool OUT = decltype(out_tag)::value, GATE = decltype(gate_tag)::value;
                const unsigned char *next = smem + (k + 1) % S::NST * S::STAGE;
                const unsigned char *last = smem + (k + S::NST - 1) % S::NST * S::STAGE;
                const bool rows_mine = PR * RS == 128 || r0 < RS, quads_mine = QR * QS == 128 || rq < QS;
                float x[IT][2], d[IT][2], o[IT][2], xo[IT][2], zo[IT][2];
                float4 v[2][QT];
                if (PREP && rows_mine) {
#pragma unroll
                    for (int i = 0; i < IT; i++) {
                        const int r = r0 + i * RS;
                        const unsigned char *p = next + r * PITCHX + ch * E;
                        get_pair<T>(p + (vec16 ? 0 : rest(px, bx, (k + 1u) * TT + r)), vec16, x[i][0], x[i][1]);
                        get_pair<T>(p + S::X_BYTES + (vec16 ? 0 : rest(pdt, bdt, (k + 1u) * TT + r)), vec16, d[i][0], d[i][1]);
                    }
                }
                if (PREP && quads_mine) {
#pragma unroll
                    for (int which = 0; which < (WITH_C ? 2 : 1); which++)
#pragma unroll
                        for (int i = 0; i < QT; i++) {
                            const int r = rq + i * QS;
                            const unsigned char *p = next + 3 * S::X_BYTES + which * S::N_BYTES + n4 * E + r * PITCHN;
                            if (!vec16n) p += which ? rest(pc, bc, (k + 1u) * TT + r) : rest(pb, bb, (k + 1u) * TT + r);
                            get_pair<T>(p, vec16n, v[which][i].x, v[which][i].y);
                            get_pair<T>(p + 2 * E, vec16n, v[which][i].z, v[which][i].w);
                        }
                }
                if (OUT && rows_mine) {
                    const float *out = at_out(k + 1) + ch * LPC;   // of tile k - 1
#pragma unroll
                    for (int i = 0; i < IT; i++) {
                        const float *p = out + (r0 + i * RS) * CH * LPC;
                        if constexpr (LPC == 1) {
                            const float2 w = *reinterpret_cast<const float2 *>(p);
                            o[i][0] = w.x, o[i][1] = w.y;
                        } else if constexpr (LPC == 2) {
                            const float4 w = *reinterpret_cast<const float4 *>(p);
                            o[i][0] = w.x + w.y, o[i][1] = w.z + w.w;
                        } else {
#pragma unroll
                            for (int c = 0; c < 2; c++) {
                                o[i][c] = 0.0f;
#pragma unroll
                                for (int j = 0; j < LPC; j += 4) {
                                    const float4 w = *reinterpret_cast<const float4 *>(p + c * LPC + j);
                                    const float sum = (w.x + w.y) + (w.z + w.w);
                                    o[i][c] = j == 0 ? sum : o[i][c] + sum;
                                }
                            }
                        }
                        const int r = r0 + i * RS;
                        const unsigned char *q = last + r * PITCHX + ch * E;
                        get_pair<T>(q + (vec16 ? 0 : rest(px, bx, (k - 1u) * TT + r)), vec16, xo[i][0], xo[i][1]);
                        if (GATE)
                            get_pair<T>(q + 2 * S::X_BYTES + (vec16 ? 0 : rest(pz, bz, (k - 1u) * TT + r)), vec16, zo[i][0], zo[i][1]);
                    }
                }
                if (rows_mine) {
                    if (PREP) {
#pragma unroll
                        for (int i = 0; i < IT; i++) {
                            d[i][0] += bias[0], d[i][1] += bias[1];
                            float p[2] = {d[i][0], d[i][1]};
                            softplus2(p[0], p[1]);
                            d[i][0] = a.softplus ? p[0] : d[i][0], d[i][1] = a.softplus ? p[1] : d[i][1];
                        }
                    }
                    if (OUT) {
#pragma unroll
                        for (int i = 0; i < IT; i++)
#pragma unroll
                            for (int c = 0; c < 2; c++) {
                                o[i][c] = a.skip ? fmaf(skip[c], xo[i][c], o[i][c]) : o[i][c];
                                if (GATE) o[i][c] *= silu(zo[i][c]);
                            }
                    }
                    if (PREP) {
                        float2 *du = at_du(k + 1);
#pragma unroll
                        for (int i = 0; i < IT; i++)
                            *reinterpret_cast<float4 *>(du + (r0 + i * RS) * CH + ch) =
                                make_float4(d[i][0], d[i][0] * x[i][0], d[i][1], d[i][1] * x[i][1]);
                    }
                }
                if (PREP && quads_mine) {
                    float *to = at_bc(k + 1);
#pragma unroll
                    for (int which = 0; which < (WITH_C ? 2 : 1); which++)
#pragma unroll
                        for (int i = 0; i < QT; i++) {
                            float4 w = v[which][i];
                            if (PAD) {   // padding states: nothing in, nothing out
                                w.x = n4 < a.n ? w.x : 0.0f, w.y = n4 + 1 < a.n ? w.y : 0.0f;
                                w.z = n4 + 2 < a.n ? w.z : 0.0f, w.w = n4 + 3 < a.n ? w.w : 0.0f;
                            }
                            *reinterpret_cast<float4 *>(to + (rq + i * QS) * 2 * NP + which * NP + n4) = w;
                        }
                }
                if (OUT && k > 0 && rows_mine) {
                    const int left = t1 - t0 - (k - 1) * TT;
#pragma unroll
                    for (int i = 0; i < IT; i++)
                        if (r0 + i * RS < left)
                            store_pair<T>(py + ((long long)(k - 1) * TT + i * RS) * a.ld_y, o[i][0], o[i][1], have, a.vec2);
                }
            };
            // Tile k is scanned while tile k + 1 is prepared and tile k - 1 finished; tile k + 2 has
            // arrived at the end of that, tile k + 3 is on its way into the place of tile k - 2.
            auto serve = [&](auto out_tag, auto gate_tag) {
                constexpr bool OUT = decltype(out_tag)::value;
                sx = px + rx * bx + qx, sdt = pdt + rx * bdt + qx, sz = pz + rx * bz + qx;
                sb = pb + rn * bb + qn, sc = pc + rn * bc + qn;
                for (int k = 0; k < 3; k++) stage(k, OUT);
                cp_wait<1>();                       // tiles 0 and 1
                helpers_sync();
                const std::true_type yes;
                const std::false_type no;
                if (tiles > 0) serve_tile(yes, out_tag, no, no, -1);
                __syncthreads();
                for (int k = 0; k < tiles; k++) {
                    stage(k + 3, OUT);
                    serve_tile(yes, out_tag, out_tag, gate_tag, k);
                    cp_wait<1>();                   // tile k + 2
                    __syncthreads();
                }
                if constexpr (OUT)
                    if (tiles > 0) serve_tile(no, no, out_tag, gate_tag, tiles);
            };
            if constexpr (SPLIT) {
                if (rank + 1 < parts) serve(std::false_type{}, std::false_type{});
                cluster_sync();
            }
            if (a.z) serve(std::true_type{}, std::true_type{});
            else serve(std::true_type{}, std::false_type{});
        };
        if (a.vec16 && a.vec16n) help(std::true_type{}, std::true_type{});
        else if (a.vec16) help(std::true_type{}, std::false_type{});
        else help(std::false_type{}, std::false_type{});
    }
    if constexpr (SPLIT) cluster_sync();   // the others may still be reading this block's part
}

// Shared memory of a block of one shape.
template <typename T> constexpr int scan_smem(int spt, int lpc) {
    const int ch = 128 / lpc, np = spt * lpc, tt = scan_rows(ch, np), e = (int)sizeof(T);
    return 5 * tt * (3 * row_pitch(ch * e) + 2 * row_pitch(np * e)) + 2 * tt * (ch * 8 + np * 8 + 128 * 4);
}

// Launches the kernel of one shape; `parts` blocks of a cluster share a sequence.
template <typename T, int SPT, int LPC, int PAD>
cudaError_t launch_scan_shape(ScanArgs a, int parts, cudaStream_t st) {
    typedef ScanShape<T, SPT, LPC> S;
    static_assert(S::SMEM == scan_smem<T>(SPT, LPC), "");
    static std::atomic<unsigned long long> attr_ctx[2];
    a.blocks = (a.cpg - 1) / S::CH + 1;
    const long long sequences = (long long)a.q.n_seq * a.groups * a.blocks;   // below 2^61
    if (sequences > 0x7FFFFFFFLL / parts) return cudaErrorInvalidConfiguration;
    const long long grid = sequences * parts;
    const int smem = S::SMEM + (parts > 1 ? S::JOIN : 0);
    void (*kernel)(ScanArgs) = parts > 1 ? scan_kernel<T, SPT, LPC, PAD, true>
                                         : scan_kernel<T, SPT, LPC, PAD, false>;
    if (smem > 48 * 1024) {   // raised once per context, as for the tensor-core kernels
        std::atomic<unsigned long long> &known = attr_ctx[parts > 1];
        const unsigned long long ctx = fcm_current_ctx_id();
        if (ctx == 0 || known.load(std::memory_order_relaxed) != ctx) {
            const cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            known.store(ctx, std::memory_order_relaxed);
        }
    }
    return launch(kernel, dim3((unsigned)grid), S::NT, (size_t)smem, st, a, parts);
}

// Shapes by states per thread and lanes per channel (seq_scan_inst_*.cu).
template <typename T> cudaError_t launch_scan(const ScanArgs &a, int spt, int lpc, int parts, cudaStream_t st);

#define FCM_SCAN_INSTANTIATE(T)                                                                      \
    template <>                                                                                      \
    cudaError_t launch_scan<T>(const ScanArgs &a, int spt, int lpc, int parts, cudaStream_t st) {    \
        const int pad = a.n == spt * lpc ? 0 : a.n % spt == 0 ? 1 : 2;                               \
        switch (spt * 256 + lpc * 4 + pad) {                                                         \
            FCM_SCAN_CASE(T, 4, 1, 0) FCM_SCAN_CASE(T, 4, 2, 0) FCM_SCAN_CASE(T, 4, 4, 0)            \
            FCM_SCAN_CASE(T, 4, 8, 0) FCM_SCAN_CASE(T, 8, 8, 0) FCM_SCAN_CASE(T, 8, 16, 0)           \
            FCM_SCAN_CASE(T, 8, 2, 0) FCM_SCAN_CASE(T, 8, 4, 0) FCM_SCAN_CASE(T, 16, 1, 0)           \
            FCM_SCAN_CASE(T, 4, 4, 1) FCM_SCAN_CASE(T, 4, 8, 1) FCM_SCAN_CASE(T, 8, 8, 1)            \
            FCM_SCAN_CASE(T, 8, 16, 1)                                                               \
            FCM_SCAN_CASE(T, 4, 1, 2) FCM_SCAN_CASE(T, 4, 2, 2) FCM_SCAN_CASE(T, 4, 4, 2)            \
            FCM_SCAN_CASE(T, 4, 8, 2) FCM_SCAN_CASE(T, 8, 8, 2) FCM_SCAN_CASE(T, 8, 16, 2)           \
        }                                                                                            \
        return cudaErrorInvalidValue;                                                                \
    }
#define FCM_SCAN_CASE(T, SPT, LPC, PAD) \
    case SPT * 256 + LPC * 4 + PAD: return launch_scan_shape<T, SPT, LPC, PAD>(a, parts, st);

}  // namespace seq
}  // namespace fcm
