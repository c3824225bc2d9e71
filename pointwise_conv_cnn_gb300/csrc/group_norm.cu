// group_norm.cu -- group normalisation with an activation and a gate, channels last.
//
//     y = act(s[d] * (x - mean) / sqrt(var + eps) + b[d]) * silu(z)
//
// Two kernels: rows that are normalised each by itself (one pixel), whose groups a few lanes hold, and
// samples of many pixels, which a cluster of blocks holds.
#include <atomic>

#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct NormArgs {
    const void *x, *z;
    const float *s, *b;
    void *y;
    long long ld_x, ld_z, ld_y, pixels;
    int n, c, cpg, groups, act, rms;
    float eps;
    int cb, nb;       // channels of a block, blocks of channels
    long long ppc;    // pixels of a block
    int hold;         // pixels that it keeps in shared memory, whole rounds of its threads
    int async;        // there is room for 8 of a thread's pixels, or for all
    int parts;        // > 0: sums only; clusters of a sample, each of which leaves its groups' sums at the sample's begin in y
    long long skip;   // pixels that hold them, behind a count of the blocks that have read them
};

// V channels at once (element by element into the vector, in place, they would be stored one by one).
template <typename T, int V> __device__ __forceinline__ void store_channels(T *p, const float (&v)[V]) {
    Vec<T, V> r;
    r.put(v);
    if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&r);
    else *reinterpret_cast<Vec<T, V> *>(p) = r;
}
// The activation and the gate; what they are is asked once for V channels.
template <int V> __device__ __forceinline__ void finish_channels(float (&v)[V], int act, bool gate, const float (&z)[V]) {
    if (act == FCM_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; i++) v[i] = silu(v[i]);
    } else if (act != FCM_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < V; i++) asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(v[i]));   // NaN stays
        if (act == FCM_ACT_RELU6)
#pragma unroll
            for (int i = 0; i < V; i++) asm("min.NaN.f32 %0, %0, 0f40C00000;" : "+f"(v[i]));
    }
    if (gate) {
#pragma unroll
        for (int i = 0; i < V; i++) v[i] *= silu(z[i]);
    }
}
// V of s or b from channel d on, a multiple of V (16-byte aligned where V >= 4), or the value that stands for none.
template <int V> __device__ __forceinline__ void load_affine(const float *p, int d, float none, float (&v)[V]) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 x = p ? *reinterpret_cast<const float4 *>(p + d + i) : make_float4(none, none, none, none);
            v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) v[i] = p ? p[d + i] : none;
    }
}
// Channels d .. d + V - 1's mean and factor, by their groups'.
template <int V, typename F> __device__ __forceinline__ void by_group(int d, int cpg, F f) {
    int g = d / cpg, left = (g + 1) * cpg - d;
#pragma unroll
    for (int i = 0; i < V; i++) {
        f(i, g);
        if (--left == 0) g++, left = cpg;
    }
}

// ---------------------------------------------------------------------------------- rows
// One pixel: LPG lanes hold a row's group, NV times V channels each, and sum it twice in registers: its
// mean, then the squares about it.  A thread has the same group of ROWS rows, all on their way at once, with
// s and b read once.  Bound by memory: 8192 rows of 32 heads of 128 with a gate, 201 MB in 42.5 us, 4.7 TB/s, 0.70 of a
// plain copy's rate.
template <typename T, int V, int LPG, int NV, int ROWS>
__global__ void __launch_bounds__(256) norm_rows_kernel(const NormArgs a) {
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const unsigned unit = blockIdx.x * (256u / LPG) + threadIdx.x / LPG;   // groups of ROWS rows: 2^31 at most, and a block's
    const int lane = threadIdx.x % LPG;
    const int g = (int)(unit % (unsigned)a.groups);
    const long long r0 = (long long)(unit / (unsigned)a.groups) * ROWS;   // past the last row: the lanes go along, and store nothing
    float x[ROWS][NV][V];
    bool in[NV];
    int d[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = (i * LPG + lane) * V;
        in[i] = e < a.cpg;
        d[i] = g * a.cpg + (in[i] ? e : 0);
    }
    Vec<T, V> raw[ROWS][NV], gate[ROWS][NV];
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
        const long long row = min(r0 + r, (long long)a.n - 1);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            raw[r][i] = *reinterpret_cast<const Vec<T, V> *>(static_cast<const T *>(a.x) + row * a.ld_x + d[i]);
            if (a.z) gate[r][i] = *reinterpret_cast<const Vec<T, V> *>(static_cast<const T *>(a.z) + row * a.ld_z + d[i]);
        }
    }
    const float inv = 1.0f / (float)a.cpg;
    float mean[ROWS], rstd[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; r++) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            raw[r][i].get(x[r][i]);
#pragma unroll
            for (int e = 0; e < V; e++) sum += in[i] ? x[r][i][e] : 0.0f;
        }
        mean[r] = 0.0f;
        if (!a.rms) {
#pragma unroll
            for (int m = LPG / 2; m; m >>= 1) sum += __shfl_xor_sync(~0u, sum, m);
            mean[r] = sum * inv;
        }
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < V; e++) {
                x[r][i][e] -= mean[r];
                sq = in[i] ? fmaf(x[r][i][e], x[r][i][e], sq) : sq;
            }
#pragma unroll
        for (int m = LPG / 2; m; m >>= 1) sq += __shfl_xor_sync(~0u, sq, m);
        rstd[r] = rsqrtf(sq * inv + a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (!in[i]) continue;
        float s[V], b[V];
        load_affine<V>(a.s, d[i], 1.0f, s);
        load_affine<V>(a.b, d[i], 0.0f, b);
#pragma unroll
        for (int r = 0; r < ROWS; r++) {
            if (r0 + r >= a.n) continue;
            float v[V], z[V] = {};
            if (a.z) gate[r][i].get(z);
#pragma unroll
            for (int e = 0; e < V; e++) v[e] = fmaf(x[r][i][e] * rstd[r], s[e], b[e]);
            finish_channels<V>(v, a.act, a.z != nullptr, z);
            store_channels<T, V>(static_cast<T *>(a.y) + (r0 + r) * a.ld_y + d[i], v);
        }
    }
}

// ---------------------------------------------------------------------------------- maps
__device__ __forceinline__ uint32_t norm_cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t norm_cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void norm_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void norm_cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void norm_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float norm_ld_cluster(uint32_t local, uint32_t rank) {
    uint32_t addr;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(~0u, v, m);
    return v;
}

template <int BYTES> __device__ __forceinline__ void norm_copy(void *to, const void *from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(to)), "l"(from), "n"(BYTES) : "memory");
}

// Sums of V channels about a first value each, of which a large mean costs the squares nothing.
template <int V> struct ChannelSums {
    float shift[V] = {}, sum[V] = {}, sq[V] = {};
    __device__ __forceinline__ void start(const float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; i++) shift[i] = v[i];
    }
    __device__ __forceinline__ void add(const float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float d = v[i] - shift[i];
            sum[i] += d, sq[i] = fmaf(d, d, sq[i]);
        }
    }
    // means in `shift`, squares about them in `sq`, of n values each
    __device__ __forceinline__ void finish(int n, bool rms) {
        const float w = 1.0f / n;
#pragma unroll
        for (int i = 0; i < V; i++) {
            if (rms) continue;   // as they are: the sums about 0
            const float q = fmaf(-sum[i] * w, sum[i], sq[i]);
            shift[i] = fmaf(sum[i], w, shift[i]), sq[i] = q < 0.0f ? 0.0f : q;
        }
    }
    // joins 2^LEVELS neighbours each, all of n values
    __device__ __forceinline__ void join(int each, float n) {
#pragma unroll
        for (int s = 1; s < V; s *= 2) {
            if (each < 2 * s) break;
#pragma unroll
            for (int i = 0; i + s < V; i += 2 * s) {
                const float d = shift[i] - shift[i + s];
                sq[i] += fmaf(0.5f * n * s * d, d, sq[i + s]);
                shift[i] = 0.5f * (shift[i] + shift[i + s]);
            }
        }
    }
};

// Normalises a thread's pixels, `step` elements apart, the first `hold` of them from shared memory; U on their way.
template <typename T, int V, int U, bool GATE>
__device__ __forceinline__ void apply_rows(int n, int hold, const T *x, long long x_step, const T *kept, int k_step, const T *z,
                                           long long z_step, T *y, long long y_step, const float (&m)[V], const float (&f)[V],
                                           const float (&b)[V], int act) {
#pragma unroll 1
    for (int i = 0; i < n; i += U) {
        Vec<T, V> raw[U], gate[GATE ? U : 1];
#pragma unroll
        for (int u = 0; u < U; u++)
            if (i + u < n) {
                raw[u] = i + u < hold ? *reinterpret_cast<const Vec<T, V> *>(kept) : *reinterpret_cast<const Vec<T, V> *>(x);
                kept += k_step, x += x_step;
                if (GATE) gate[u] = *reinterpret_cast<const Vec<T, V> *>(z), z += z_step;
            }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (i + u < n) {
                float v[V], zv[V] = {};
                raw[u].get(v);
                if (GATE) gate[u].get(zv);
#pragma unroll
                for (int k = 0; k < V; k++) v[k] = fmaf(v[k] - m[k], f[k], b[k]);
                finish_channels<V>(v, act, GATE, zv);
                store_channels<T, V>(y, v);
                y += y_step;
            }
    }
}

// Where a shared sample's sums wait in its outputs: the first 16-byte boundary.
__device__ __forceinline__ float *sums_of(void *y) {
    return reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(y) + 15) & ~(uintptr_t)15);
}

// N lanes' counts, means and squares about the mean as those of all their values, in every lane; a count of 0 says nothing.
template <int N> __device__ __forceinline__ void join_sums(float &n, float &m, float &q) {
    float total = n, sum = n > 0.0f ? n * m : 0.0f;
#pragma unroll
    for (int s = N / 2; s; s >>= 1) total += __shfl_xor_sync(~0u, total, s), sum += __shfl_xor_sync(~0u, sum, s);
    const float mean = __fdividef(sum, total), d = m - mean;
    q = n > 0.0f ? fmaf(n * d, d, q) : 0.0f;
#pragma unroll
    for (int s = N / 2; s; s >>= 1) q += __shfl_xor_sync(~0u, q, s);
    n = total, m = mean;
}

// Many pixels: a cluster has a sample's block of channels (whole groups), each of its blocks a share of the
// pixels, which it keeps in shared memory as far as they fit, so that x comes from memory once; the rest is
// read again (from the L2).  A thread has V channels of every TY-th pixel, which it brings to shared memory itself, 8
// on their way at once, and reads there: no registers wait for memory, and no barrier.  The pixels that are not kept go
// first, through the places that the last kept ones will have.  Sums are joined by their counts, means and squares
// about the mean: a thread's channels of a group, threads in shared memory, blocks through distributed shared memory,
// in one order always.
constexpr int kMapThreads = 256;
template <typename T, int V, bool GATE, int BLOCKS> __global__ void __launch_bounds__(kMapThreads, BLOCKS) norm_maps_kernel(const NormArgs a) {
    constexpr int U = BLOCKS == 2 ? 4 : 2, RING = 8, nt = kMapThreads, warps = nt / 32;
    constexpr int BYTES = V * sizeof(T);
    constexpr bool ASYNC = BYTES >= 4;   // single 16-bit channels go through registers
    extern __shared__ __align__(16) unsigned char smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float *part_m = reinterpret_cast<float *>(smem), *part_q = part_m + nt * V;   // [TY][a pass's channels, joined]
    float *group = part_q + nt * V;   // count, mean, squares of this block's groups, then mean and factor of the cluster's
    const int gb = a.cb / a.cpg;
    T *kept = reinterpret_cast<T *>(group + (5 * gb + 3) / 4 * 4);
    const uint32_t ranks = norm_cluster_size(), rank = norm_cluster_rank();
    const int parts = max(a.parts, 1), cluster = (int)(blockIdx.x / ranks), part = cluster % parts;
    const int block = cluster / parts % a.nb, sample = cluster / parts / a.nb;
    const int c0 = block * a.cb, cc = min(a.cb, a.c - c0), cols = cc / V, groups = cc / a.cpg;
    const long long p0 = min((long long)(part * ranks + rank) * a.ppc, a.pixels), p1 = min(p0 + a.ppc, a.pixels);
    const int np = (int)(p1 - p0);
    const int cw = min(a.cb / V, nt), ty_n = nt / cw, tx = threadIdx.x % cw, ty = threadIdx.x / cw;
    const int rows = min(np, ty_n), full = np / ty_n, extra = np % ty_n;   // thread rows with pixels, their counts
    const int mine = ty < ty_n ? full + (ty < extra) : 0, hold = min(mine, a.hold / ty_n), passing = mine - hold;
    const int each = a.cpg % V == 0 ? V : V % a.cpg == 0 ? a.cpg : 1, entries = V / each;   // channels joined in a thread
    const long long first = (long long)sample * a.pixels + p0;
    const T *x = static_cast<const T *>(a.x) + first * a.ld_x + c0;
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    for (int i = threadIdx.x; i < 3 * gb; i += nt) group[i] = 0.0f;
    for (int k0 = 0; k0 < cols; k0 += cw) {
        const int kw = min(cw, cols - k0), col = k0 + tx;
        __syncthreads();
        if (mine > 0 && tx < kw) {
            ChannelSums<V> s;
            // the thread's i-th pixel: passing ones first, in the places of kept ones; its place there
            auto pixel = [&](int i) { return ty + (i < passing ? hold + i : i - passing) * ty_n; };
            auto place = [&](int i) {
                const int at = i < passing ? (i - passing) & (RING - 1) : i - passing;   // RING divides 2^32
                return kept + ((size_t)(ty + at * ty_n) * cols + col) * V;
            };
            bool done = false;
            if constexpr (ASYNC)
                if (a.async) {
                    T *const to = kept + ((size_t)ty * cols + col) * V;
                    const int round = ty_n * cols * V;
                    auto at = [&](int i) { return to + (i < passing ? (i - passing) & (RING - 1) : i - passing) * round; };
                    const T *kept_from = x + (long long)ty * a.ld_x + col * V, *from = kept_from + (long long)hold * ty_n * a.ld_x;
                    const long long step = ty_n * a.ld_x;
                    if (passing == 0) from = kept_from;
#pragma unroll 1
                    for (int i = -RING; i < mine; i++) {
                        if (i >= 0) {
                            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
                            float v[V];
                            reinterpret_cast<const Vec<T, V> *>(at(i))->get(v);
                            if (i == 0 && !a.rms) s.start(v);
                            s.add(v);
                        }
                        if (i + RING < mine) norm_copy<BYTES>(at(i + RING), from);
                        from = i + RING + 1 == passing ? kept_from : from + step;
                        asm volatile("cp.async.commit_group;" ::: "memory");
                    }
                    done = true;
                }
            if (!done) {
#pragma unroll 1
                for (int i = 0; i < mine; i += U) {
                    Vec<T, V> raw[U];
                    const int have = min(U, mine - i);
#pragma unroll
                    for (int u = 0; u < U; u++)
                        if (u < have) raw[u] = *reinterpret_cast<const Vec<T, V> *>(x + (long long)pixel(i + u) * a.ld_x + col * V);
#pragma unroll
                    for (int u = 0; u < U; u++)
                        if (u < have) {
                            if (i + u >= passing) *reinterpret_cast<Vec<T, V> *>(place(i + u)) = raw[u];
                            float v[V];
                            raw[u].get(v);
                            if (i + u == 0 && !a.rms) s.start(v);
                            s.add(v);
                        }
                }
            }
            s.finish(mine, a.rms);
            s.join(each, (float)mine);
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i % each == 0) {
                    part_m[(ty * kw + tx) * entries + i / each] = s.shift[i];
                    part_q[(ty * kw + tx) * entries + i / each] = s.sq[i];
                }
        }
        __syncthreads();
        // the pass's channels [k0 * V, (k0 + kw) * V) of each group, by a warp: over the rows' lanes where there are many
        for (int g = k0 * V / a.cpg + warp; g < groups && g * a.cpg < (k0 + kw) * V; g += warps) {
            const int from = max(g * a.cpg, k0 * V) - k0 * V, to = min((g + 1) * a.cpg, (k0 + kw) * V) - k0 * V;
            const int e0 = from / each, width = (to - from) / each, pitch = kw * entries;
            const bool tall = rows >= width;
            const int r_first = tall ? lane : 0, r_step = tall ? 32 : 1, k_first = tall ? 0 : lane, k_step = tall ? 1 : 32;
            float n = 0.0f, m = 0.0f;
            for (int r = r_first; r < rows; r += r_step) {
                const float count = (float)((full + (r < extra)) * each);
                for (int k = k_first; k < width; k += k_step) n += count, m = fmaf(count, part_m[r * pitch + e0 + k], m);
            }
            n = warp_sum(n), m = warp_sum(m);
            const float mean = n > 0.0f ? m / n : 0.0f;
            float q = 0.0f;
            for (int r = r_first; r < rows; r += r_step) {
                const float count = (float)((full + (r < extra)) * each);
                for (int k = k_first; k < width; k += k_step) {
                    const float d = part_m[r * pitch + e0 + k] - mean;
                    q += fmaf(count * d, d, part_q[r * pitch + e0 + k]);
                }
            }
            q = warp_sum(q);
            if (lane == 0 && n > 0.0f) {
                float *have = group + 3 * g;
                const float total = have[0] + n, d = mean - have[1];
                have[2] += q + d * d * (have[0] * n / total);
                have[1] += d * (n / total);
                have[0] = total;
            }
        }
    }
    __syncthreads();
    if (ranks > 1) norm_cluster_sync();
    // the cluster's groups: a lane has a block's sums, 16 a group
    float *mean_of = group + 3 * gb, *factor_of = mean_of + gb;
    for (int g0 = 2 * warp; g0 < groups; g0 += 2 * warps) {
        const int g = min(g0 + lane / 16, groups - 1);
        const uint32_t at = tc::smem_u32(group + 3 * g), from = lane % 16;
        float n = 0.0f, m = 0.0f, q = 0.0f;
        if (from < ranks) n = norm_ld_cluster(at, from), m = norm_ld_cluster(at + 4, from), q = norm_ld_cluster(at + 8, from);
        join_sums<16>(n, m, q);
        if (from == 0) {
            if (!a.parts) {
                mean_of[g] = a.rms ? 0.0f : m, factor_of[g] = rsqrtf(__fdividef(q, n) + a.eps);
            } else if (rank == 0) {
                float *begin = sums_of(static_cast<T *>(a.y) + (long long)sample * a.pixels * a.c);
                float *to = begin + 4 + 3 * ((long long)part * a.groups + g);
                to[0] = n, to[1] = m, to[2] = q;
                if (part == 0 && g == 0) *reinterpret_cast<unsigned *>(begin) = 0;
            }
        }
    }
    __syncthreads();
    if (ranks > 1) norm_cluster_arrive();   // waited for at the end: the others may still read this block's sums
    if (a.parts) {
        if (ranks > 1) norm_cluster_wait();
        return;
    }
    T *y = static_cast<T *>(a.y) + first * a.ld_y + c0;
    const T *z = a.z ? static_cast<const T *>(a.z) + first * a.ld_z + c0 : nullptr;
    for (int k0 = 0; k0 < cols; k0 += cw) {
        const int col = k0 + tx;
        if (ty >= ty_n || col >= cols) continue;
        float m[V], f[V], b[V];
        load_affine<V>(a.s, c0 + col * V, 1.0f, f);
        load_affine<V>(a.b, c0 + col * V, 0.0f, b);
        by_group<V>(col * V, a.cpg, [&](int i, int g) { m[i] = mean_of[g], f[i] *= factor_of[g]; });
        const T *xp = x + (long long)ty * a.ld_x + col * V, *zp = z ? z + (long long)ty * a.ld_z + col * V : nullptr;
        T *yp = y + (long long)ty * a.ld_y + col * V;
        const T *kp = kept + ((size_t)ty * cols + col) * V;
        const long long x_step = ty_n * a.ld_x, z_step = ty_n * a.ld_z, y_step = ty_n * a.ld_y;
        const int k_step = ty_n * cols * V;
        apply_rows<T, V, U, GATE>(mine, hold, xp, x_step, kp, k_step, zp, z_step, yp, y_step, m, f, b, a.act);
    }
    __syncwarp();
    if (ranks > 1) norm_cluster_wait();
}

// The second step of samples that clusters share (run_shared): their sums joined, the pixels normalised.  The block that
// is the last to have read a sample's sums also writes the pixels that they lie in.  512 x 512 x 128 bf16: 25 us for the
// sums (2.6 TB/s) and 30 for this (4.5 TB/s of x and y); two rounds of blocks, which all join the sums first, took 38.
template <typename T, int V, bool GATE> __global__ void __launch_bounds__(256, 2) norm_apply_kernel(const NormArgs a) {
    extern __shared__ float stats[];   // mean and factor of each group
    __shared__ bool last;
    const int cols = a.c / V, nt = 256, cw = min(cols, nt), ty_n = nt / cw, tx = threadIdx.x % cw, ty = threadIdx.x / cw;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int sample = blockIdx.x / a.nb, block = blockIdx.x % a.nb;   // nb: blocks of a sample
    const long long begin = (long long)sample * a.pixels;
    const long long p0 = a.skip + block * a.ppc, p1 = min(p0 + a.ppc, a.pixels);
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    float *sums = sums_of(static_cast<T *>(a.y) + begin * a.c) + 4;
    // a warp's next group is on its way while one is joined
    auto load = [&](int g, float (&v)[3]) {
        const float *p = sums + 3 * ((long long)min(lane, a.parts - 1) * a.groups + min(g, a.groups - 1));
        v[0] = p[0], v[1] = p[1], v[2] = p[2];
    };
    float v[3], w[3];
    load(warp, v);
#pragma unroll 1
    for (int g = warp; g < a.groups; g += 8) {
        load(g + 8, w);
        float n = lane < a.parts ? v[0] : 0.0f, m = v[1], q = v[2];
        join_sums<32>(n, m, q);
        if (lane == 0) stats[2 * g] = a.rms ? 0.0f : m, stats[2 * g + 1] = rsqrtf(__fdividef(q, n) + a.eps);
#pragma unroll
        for (int i = 0; i < 3; i++) v[i] = w[i];
    }
    __syncthreads();
    if (threadIdx.x == 0) {   // all of this block's reads are done
        __threadfence();
        last = atomicAdd(reinterpret_cast<unsigned *>(sums) - 4, 1u) == (unsigned)a.nb - 1;
    }
    const T *x = static_cast<const T *>(a.x) + begin * a.ld_x, *z = a.z ? static_cast<const T *>(a.z) + begin * a.ld_z : nullptr;
    T *y = static_cast<T *>(a.y) + begin * a.c;
    auto normalise = [&](long long p0, long long p1) {
        const int mine = p1 - p0 > ty ? (int)((p1 - p0 - ty + ty_n - 1) / ty_n) : 0;
        for (int col = tx; ty < ty_n && col < cols; col += cw) {
            float m[V], f[V], b[V];
            load_affine<V>(a.s, col * V, 1.0f, f);
            load_affine<V>(a.b, col * V, 0.0f, b);
            by_group<V>(col * V, a.cpg, [&](int i, int g) { m[i] = stats[2 * g], f[i] *= stats[2 * g + 1]; });
            const T *xp = x + (p0 + ty) * a.ld_x + col * V, *zp = GATE ? z + (p0 + ty) * a.ld_z + col * V : nullptr;
            T *yp = y + (p0 + ty) * a.c + col * V;
            apply_rows<T, V, 4, GATE>(mine, 0, xp, ty_n * a.ld_x, xp, 0, zp, ty_n * a.ld_z, yp, (long long)ty_n * a.c, m, f, b, a.act);
        }
    };
    __syncthreads();
    const int turns = last ? 2 : 1;
    __threadfence();
#pragma unroll 1   // one copy of the code
    for (int turn = 0; turn < turns; turn++) normalise(turn ? 0 : p0, turn ? a.skip : p1);
}

// Bytes of shared memory beside the kept pixels.
template <int V> static size_t maps_fixed(int groups_of_block) {
    return (size_t)kMapThreads * V * 8 + (size_t)(5 * groups_of_block + 3) / 4 * 16;
}

template <typename T, int V, int BLOCKS>
static cudaError_t launch_maps(const NormArgs &a, long long blocks, size_t smem, int cl, cudaStream_t st) {
    static std::atomic<unsigned long long> attr{0};
    const unsigned long long ctx = fcm_current_ctx_id();
    void (*const plain)(NormArgs) = norm_maps_kernel<T, V, false, BLOCKS>;
    void (*const gated)(NormArgs) = norm_maps_kernel<T, V, true, BLOCKS>;
    if (ctx == 0 || attr.load(std::memory_order_relaxed) != ctx) {
        cudaError_t e = cudaFuncSetAttribute(plain, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(gated, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        attr.store(ctx, std::memory_order_relaxed);
    }
    return launch(a.z ? gated : plain, dim3((unsigned)blocks), kMapThreads, smem, st, a, cl);
}

// Samples too large for a cluster: clusters share one, and leave their groups' sums in y's first pixels, which are written
// when all have read them.  So whole rows are read and written, by all SMs, and no memory is needed beside the caller's.
constexpr int kMostParts = 32;
template <typename T, int V> static cudaError_t run_shared(NormArgs a, int sms, cudaStream_t st) {
    constexpr int CL = 8, NT = kMapThreads;
    a.cb = a.c;
    const int cols = a.c / V, round = NT / (cols < NT ? cols : NT);
    const size_t fixed = maps_fixed<V>(a.groups), ring = (size_t)8 * round * a.c * sizeof(T), stats = (size_t)8 * a.groups;
    a.async = fixed + ring <= 110 * 1024;
    a.hold = a.async ? 8 * round : 0;
    const long long row = a.c * (long long)sizeof(T);
    const int parts = 4 * sms / CL / a.n;
    a.parts = parts < 1 ? 1 : parts > kMostParts ? kMostParts : parts;
    a.nb = 1;
    a.ppc = (a.pixels + a.parts * CL - 1) / (a.parts * CL);
    cudaError_t e = launch_maps<T, V, 2>(a, (long long)a.n * a.parts * CL, fixed + (a.async ? ring : 0), CL, st);
    if (e != cudaSuccess) return e;
    a.skip = (32 + 12ll * a.parts * a.groups + row - 1) / row;
    // as many blocks as are on the SMs at once: each joins the sums first
    const long long blocks = a.n < 2 * sms ? 2ll * sms / a.n : 1, rest = a.pixels - a.skip;
    a.ppc = (rest + blocks - 1) / blocks;
    a.nb = (int)((rest + a.ppc - 1) / a.ppc);
    return launch(a.z ? norm_apply_kernel<T, V, true> : norm_apply_kernel<T, V, false>, dim3((unsigned)(a.n * a.nb)), 256, stats, st, a);
}

template <typename T, int V> static cudaError_t run_maps(NormArgs a, bool may_share, int sms, cudaStream_t st) {
    // Whole vectors of whole groups.
    long long unit = a.cpg;
    while (unit % V) unit += a.cpg;
    const int units = (int)(a.c / unit);
    const size_t most = 227 * 1024 - 1024;
    int nb = 1, cl = 1;
    auto seg = [&](int blocks) { return (units + blocks - 1) / blocks * unit * (long long)sizeof(T); };   // bytes of a row
    auto piece = [&] { return (double)((a.pixels + cl - 1) / cl) * seg(nb); };
    for (;;) {
        const bool few = (long long)a.n * nb * cl < 2 * sms;
        if (!few && piece() <= 72 * 1024) break;
        if (nb < units && seg(2 * nb) >= 64) nb *= 2;
        else if (cl < 8 && a.pixels >= 16 * cl && piece() > 16 * 1024) cl *= 2;
        else if (few && nb < units && seg(2 * nb) >= 32) nb *= 2;
        else break;
    }
    // Whether clusters share samples instead, which costs two launches and the joining of their sums, some 30 us.  A block
    // takes 1.1 ns a vector and so does an SM (measured from 40000 x 66 in pairs of channels, 204 us by 8 blocks and 16 shared,
    // to 512 x 512 x 128, 55 shared).  What the blocks' shared memory does not keep is read again, at half the speed: a sample of
    // 40000 x 128 21 us and 33 shared, 90000 x 128 53 and 39; 32 samples of 8192 x 128 106 and 75, 16 32 and 51.
    const double sample = (double)a.pixels * a.c, vectors = sample / V, blocks = (double)nb * cl, bytes = sample * sizeof(T);
    if (may_share && (1.1e-3 * vectors / blocks > 35.0 + 1.1e-3 * vectors * a.n / sms || bytes > 16e6 ||
                      (bytes > 1.5e6 && bytes * a.n > 38e6)))
        return run_shared<T, V>(a, sms, st);
    const int per = (units + nb - 1) / nb;
    a.cb = (int)(per * unit), a.nb = (units + per - 1) / per;
    a.ppc = (a.pixels + cl - 1) / cl;
    const size_t fixed = maps_fixed<V>(a.cb / a.cpg), row = (size_t)a.cb * sizeof(T);
    // whole rounds of the threads' pixels, and room for 8 on their way
    const int cols = a.cb / V, round = kMapThreads / (cols < kMapThreads ? cols : kMapThreads);
    const long long rounds = (a.ppc + round - 1) / round, room = (long long)((most - fixed) / row) / round;
    a.async = room >= rounds || room >= 8;
    a.hold = (int)((rounds < room ? rounds : room) * round);
    const size_t smem = fixed + a.hold * row;
    // Three blocks an SM, with fewer registers, where there are blocks for more than two rounds of two and room for three: us with
    // two and three, 64 x 56 x 56 x 128 (1024 blocks) 44.7 and 38.5, 32 x (512) 26.0 and 28.3, 16 x 18.8 and 20.4;
    // 64 x 32 x 32 x 320 50.9 and 43.1, gated 64 x 56 x 56 x 128 in bf16 78.1 and 74.9 (seven registers of it spill).
    const long long all = (long long)a.n * a.nb * cl;
    if constexpr (V * sizeof(T) == 16)
        if (all > 4ll * sms && smem <= 74 * 1024) return launch_maps<T, V, 3>(a, all, smem, cl, st);
    return launch_maps<T, V, 2>(a, all, smem, cl, st);
}

template <typename T, int V, int LPG, int NV, int ROWS> static cudaError_t rows_kernel(const NormArgs &a, cudaStream_t st) {
    const long long units = (long long)(a.n + ROWS - 1) / ROWS * a.groups;
    return launch(norm_rows_kernel<T, V, LPG, NV, ROWS>, dim3((unsigned)((units * LPG + 255) / 256)), 256, 0, st, a);
}

template <typename T> static cudaError_t run_norm(const NormArgs &a, int sms, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = aligned16(a.x) && aligned16(a.y) && aligned16(a.z) && aligned16(a.s) && aligned16(a.b) &&
                     ((a.ld_x | a.ld_y | (a.z ? a.ld_z : 0) | a.c) % V) == 0;
    if (a.pixels == 1 && vec && a.cpg % V == 0 && a.cpg <= 128 * V) {
        const int n = a.cpg / V;
        return n <= 8    ? rows_kernel<T, V, 8, 1, 4>(a, st)
               : n <= 16 ? rows_kernel<T, V, 16, 1, 4>(a, st)
               : n <= 32 ? rows_kernel<T, V, 32, 1, 4>(a, st)
               : n <= 64 ? rows_kernel<T, V, 32, 2, 2>(a, st)
                         : rows_kernel<T, V, 32, 4, 1>(a, st);
    }
    if (a.pixels == 1 && a.cpg <= 256)
        return a.cpg <= 64 ? rows_kernel<T, 1, 32, 2, 4>(a, st) : rows_kernel<T, 1, 32, 8, 2>(a, st);
    // a shared sample's sums need room in outputs that are not inputs, and few pixels of it
    const bool may_share = a.x != a.y && a.ld_y == a.c && a.groups <= 2048 && a.pixels >= 4096;
    if (vec) return run_maps<T, V>(a, may_share, sms, st);
    if constexpr (sizeof(T) == 2) {   // two channels at once
        const auto at4 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; };
        if (at4(a.x) && at4(a.y) && at4(a.z) && ((a.ld_x | a.ld_y | (a.z ? a.ld_z : 0) | a.c) % 2) == 0)
            return run_maps<T, 2>(a, may_share, sms, st);
    }
    return run_maps<T, 1>(a, may_share, sms, st);
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_group_norm(const fcm_norm_desc *desc, const void *x, const float *s, const float *b,
                                     const void *z, void *y, void *stream) {
    FcmNvtxRange nvtx("fcm_group_norm");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_norm_desc d = *desc;
    if (d.n < 0 || d.pixels < 0 || d.c < 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "n %d, pixels %lld, c %d", d.n, d.pixels, d.c);
    if (d.groups < 1 || d.c % d.groups)
        return fcm_fail(FCM_ERR_INVALID_ARG, "%d groups do not divide %d channels", d.groups, d.c);
    if (d.dtype < FCM_F32 || d.dtype > FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d.dtype);
    if (d.act < FCM_ACT_NONE || d.act > FCM_ACT_SILU)
        return fcm_fail(FCM_ERR_INVALID_ARG, "activation code out of range");
    if (d.rms != 0 && d.rms != 1) return fcm_fail(FCM_ERR_INVALID_ARG, "rms %d: 0 or 1", d.rms);
    if (!(d.eps >= 0.0f)) return fcm_fail(FCM_ERR_INVALID_ARG, "eps %g is not at least 0", (double)d.eps);
    if (d.pixels > (1LL << 31) - 1)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "%lld pixels; at most 2^31 - 1", d.pixels);
    if (d.c > 8192) return fcm_fail(FCM_ERR_UNSUPPORTED, "%d channels; at most 8192", d.c);
    if ((long long)d.n * d.c > (1LL << 31) - 1)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "%d samples of %d channels; at most 2^31 - 1 in all", d.n, d.c);
    fcm_status st;
    if ((st = seq::check_ld(&d.ld_x, d.c, "ld_x")) != FCM_OK || (st = seq::check_ld(&d.ld_z, d.c, "ld_z")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_y, d.c, "ld_y")) != FCM_OK)
        return st;
    if (d.n == 0 || d.pixels == 0) return FCM_OK;
    const size_t e = (size_t)fcm_dtype_bytes(d.dtype);
    if ((st = seq::check_dev_ptr(x, e, "x")) != FCM_OK || (st = seq::check_dev_ptr(y, e, "y")) != FCM_OK ||
        (z && (st = seq::check_dev_ptr(z, e, "z")) != FCM_OK) || (s && (st = seq::check_dev_ptr(s, 4, "s")) != FCM_OK) ||
        (b && (st = seq::check_dev_ptr(b, 4, "b")) != FCM_OK))
        return st;
    const long long rows = d.n * d.pixels;
    if (!(x == y && d.ld_x == d.ld_y) && seq::rows_overlap(x, d.ld_x, d.c, y, d.ld_y, d.c, rows, e))
        return fcm_fail(FCM_ERR_INVALID_ARG, "x and y overlap without being the same");
    if (z && seq::rows_overlap(z, d.ld_z, d.c, y, d.ld_y, d.c, rows, e))
        return fcm_fail(FCM_ERR_INVALID_ARG, "z and y overlap");
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;

    seq::NormArgs a = {};
    a.x = x, a.z = z, a.s = s, a.b = b, a.y = y;
    a.ld_x = d.ld_x, a.ld_z = d.ld_z, a.ld_y = d.ld_y, a.pixels = d.pixels;
    a.n = d.n, a.c = d.c, a.cpg = d.c / d.groups, a.groups = d.groups, a.act = d.act, a.rms = d.rms, a.eps = d.eps;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t ce = d.dtype == FCM_F32   ? seq::run_norm<float>(a, sms, cs)
                           : d.dtype == FCM_F16 ? seq::run_norm<__half>(a, sms, cs)
                                                : seq::run_norm<__nv_bfloat16>(a, sms, cs);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
