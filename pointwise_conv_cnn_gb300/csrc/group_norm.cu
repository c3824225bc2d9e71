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
    int hold;         // pixels that it keeps in shared memory
};

template <typename T, int V> __device__ __forceinline__ void load_channels(const T *p, float (&v)[V]) {
    reinterpret_cast<const Vec<T, V> *>(p)->get(v);
}
// V of s or b from channel d on, or the value that stands for none.
template <int V> __device__ __forceinline__ void load_affine(const float *p, int d, float none, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i++) v[i] = p ? p[d + i] : none;
}

// ---------------------------------------------------------------------------------- rows
// One pixel: LPG lanes hold a row's group, NV times V channels each, and sum it twice in registers: its
// mean, then the squares about it.  A thread has the same group of ROWS rows, all on their way at once, with
// s and b read once.
template <typename T, int V, int LPG, int NV, int ROWS>
__global__ void __launch_bounds__(256) norm_rows_kernel(const NormArgs a) {
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const long long unit = ((long long)blockIdx.x * 256 + threadIdx.x) / LPG;
    const int lane = threadIdx.x % LPG;
    const int g = (int)(unit % a.groups);
    const long long r0 = unit / a.groups * ROWS;   // past the last row: the lanes go along, and store nothing
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
            float v[V], z[V];
            if (a.z) gate[r][i].get(z);
#pragma unroll
            for (int e = 0; e < V; e++) {
                v[e] = act_seq(fmaf(x[r][i][e] * rstd[r], s[e], b[e]), a.act);
                if (a.z) v[e] *= silu(z[e]);
            }
            reinterpret_cast<Vec<T, V> *>(static_cast<T *>(a.y) + (r0 + r) * a.ld_y + d[i])->put(v);
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

// Many pixels: a cluster has a sample's block of channels (whole groups), each of its blocks a share of the
// pixels, which it keeps in shared memory as far as they fit, so that x comes from memory once; the rest is
// read again (from the L2).  A thread has V channels of every TY-th pixel.  Their sums are taken about the
// mean of its first pixels, so that a large mean costs the squares nothing, and joined by their counts,
// means and squares about the mean: threads in shared memory, blocks through distributed shared memory, in
// one order always.
template <typename T, int V> __global__ void __launch_bounds__(512) norm_maps_kernel(const NormArgs a) {
    constexpr int U = 4;
    extern __shared__ __align__(16) unsigned char smem[];
    const int nt = blockDim.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = nt / 32;
    float *part_m = reinterpret_cast<float *>(smem), *part_q = part_m + nt * V;   // [TY][channels of a pass]
    float *group = part_q + nt * V;   // count, mean, squares of this block's groups, then mean and factor of the cluster's
    const int gb = a.cb / a.cpg;
    T *kept = reinterpret_cast<T *>(group + (5 * gb + 3) / 4 * 4);
    const uint32_t ranks = norm_cluster_size(), rank = norm_cluster_rank();
    const int block = (int)(blockIdx.x / ranks) % a.nb, sample = (int)(blockIdx.x / ranks) / a.nb;
    const int c0 = block * a.cb, cc = min(a.cb, a.c - c0), cols = cc / V, groups = cc / a.cpg;
    const long long p0 = min((long long)rank * a.ppc, a.pixels), p1 = min(p0 + a.ppc, a.pixels);
    const int np = (int)(p1 - p0), hold = min(np, a.hold);
    const int cw = min(cols, nt), ty_n = nt / cw, tx = threadIdx.x % cw, ty = threadIdx.x / cw;
    const long long first = (long long)sample * a.pixels + p0;
    const T *x = static_cast<const T *>(a.x) + first * a.ld_x + c0;
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    for (int i = threadIdx.x; i < 3 * gb; i += nt) group[i] = 0.0f;
    for (int k0 = 0; k0 < cols; k0 += cw) {
        const int kw = min(cw, cols - k0), col = k0 + tx;
        __syncthreads();
        if (ty < ty_n && tx < kw) {
            float shift[V] = {}, sum[V] = {}, sq[V] = {};
            int count = 0;
            for (int p = ty; p < np; p += U * ty_n) {
                Vec<T, V> raw[U];
                const int have = min(U, (np - p + ty_n - 1) / ty_n);
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (u < have) raw[u] = *reinterpret_cast<const Vec<T, V> *>(x + (long long)(p + u * ty_n) * a.ld_x + col * V);
                if (!a.rms && count == 0) {
                    const float w = 1.0f / have;
#pragma unroll
                    for (int u = 0; u < U; u++)
                        if (u < have) {
                            float v[V];
                            raw[u].get(v);
#pragma unroll
                            for (int i = 0; i < V; i++) shift[i] = fmaf(v[i], w, shift[i]);
                        }
                }
                count += have;
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (u < have) {
                        const int at = p + u * ty_n;
                        if (at < hold) *reinterpret_cast<Vec<T, V> *>(kept + ((size_t)at * cols + col) * V) = raw[u];
                        float v[V];
                        raw[u].get(v);
#pragma unroll
                        for (int i = 0; i < V; i++) {
                            const float d = v[i] - shift[i];
                            sum[i] += d, sq[i] = fmaf(d, d, sq[i]);
                        }
                    }
            }
            const float w = count ? 1.0f / count : 0.0f;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int at = (ty * kw + tx) * V + i;
                part_m[at] = a.rms ? 0.0f : fmaf(sum[i], w, shift[i]);
                part_q[at] = a.rms ? sq[i] : fmaxf(fmaf(-sum[i] * w, sum[i], sq[i]), sq[i] != sq[i] ? sq[i] : 0.0f);
            }
        }
        __syncthreads();
        // the pass's channels [k0 * V, (k0 + kw) * V) of each group, by a warp
        for (int g = k0 * V / a.cpg + warp; g < groups && g * a.cpg < (k0 + kw) * V; g += warps) {
            const int from = max(g * a.cpg, k0 * V) - k0 * V, to = min((g + 1) * a.cpg, (k0 + kw) * V) - k0 * V;
            const int width = to - from, entries = width * ty_n;
            float n = 0.0f, m = 0.0f;
            for (int e = lane; e < entries; e += 32) {
                const int r = e / width, ch = from + e % width;
                const float k = (float)((np - r + ty_n - 1) / ty_n);
                if (r < np) n += k, m = fmaf(k, part_m[r * kw * V + ch], m);
            }
            n = warp_sum(n), m = warp_sum(m);
            const float mean = n > 0.0f ? m / n : 0.0f;
            float q = 0.0f;
            for (int e = lane; e < entries; e += 32) {
                const int r = e / width, ch = from + e % width;
                if (r >= np) continue;
                const float d = part_m[r * kw * V + ch] - mean;
                q += fmaf((float)((np - r + ty_n - 1) / ty_n) * d, d, part_q[r * kw * V + ch]);
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
    float *mean_of = group + 3 * gb, *factor_of = mean_of + gb;
    for (int g = threadIdx.x; g < groups; g += nt) {
        const uint32_t at = tc::smem_u32(group + 3 * g);
        float n = 0.0f, m = 0.0f, q = 0.0f;
        for (uint32_t r = 0; r < ranks; r++) {
            const float k = norm_ld_cluster(at, r);
            n += k, m = fmaf(k, norm_ld_cluster(at + 4, r), m);
        }
        m /= n;
        for (uint32_t r = 0; r < ranks; r++) {
            const float d = norm_ld_cluster(at + 4, r) - m, k = norm_ld_cluster(at, r);
            if (k > 0.0f) q += fmaf(k * d, d, norm_ld_cluster(at + 8, r));
        }
        mean_of[g] = a.rms ? 0.0f : m;
        factor_of[g] = rsqrtf(q / n + a.eps);
    }
    __syncthreads();
    T *y = static_cast<T *>(a.y) + first * a.ld_y + c0;
    const T *z = a.z ? static_cast<const T *>(a.z) + first * a.ld_z + c0 : nullptr;
    for (int k0 = 0; k0 < cols; k0 += cw) {
        const int col = k0 + tx;
        if (ty >= ty_n || col >= cols) continue;
        float m[V], f[V], b[V];
        load_affine<V>(a.s, c0 + col * V, 1.0f, f);
        load_affine<V>(a.b, c0 + col * V, 0.0f, b);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int g = (col * V + i) / a.cpg;
            m[i] = mean_of[g], f[i] *= factor_of[g];
        }
        for (int p = ty; p < np; p += U * ty_n) {
            Vec<T, V> raw[U], gate[U];
            const int have = min(U, (np - p + ty_n - 1) / ty_n);
#pragma unroll
            for (int u = 0; u < U; u++)
                if (u < have) {
                    const int at = p + u * ty_n;
                    raw[u] = at < hold ? *reinterpret_cast<const Vec<T, V> *>(kept + ((size_t)at * cols + col) * V)
                                       : *reinterpret_cast<const Vec<T, V> *>(x + (long long)at * a.ld_x + col * V);
                    if (z) gate[u] = *reinterpret_cast<const Vec<T, V> *>(z + (long long)at * a.ld_z + col * V);
                }
#pragma unroll
            for (int u = 0; u < U; u++)
                if (u < have) {
                    float v[V], zv[V];
                    raw[u].get(v);
                    if (z) gate[u].get(zv);
#pragma unroll
                    for (int i = 0; i < V; i++) {
                        v[i] = act_seq(fmaf(v[i] - m[i], f[i], b[i]), a.act);
                        if (z) v[i] *= silu(zv[i]);
                    }
                    reinterpret_cast<Vec<T, V> *>(y + (long long)(p + u * ty_n) * a.ld_y + col * V)->put(v);
                }
        }
    }
    if (ranks > 1) norm_cluster_sync();   // the others may still read this block's sums
}

// Bytes of shared memory beside the kept pixels.
template <int V> static size_t maps_fixed(int nt, int groups_of_block) {
    return (size_t)nt * V * 8 + (size_t)(5 * groups_of_block + 3) / 4 * 16;
}

template <typename T, int V> static cudaError_t run_maps(NormArgs a, int sms, cudaStream_t st) {
    // Whole vectors of whole groups.
    long long unit = a.cpg;
    while (unit % V) unit += a.cpg;
    const int units = (int)(a.c / unit);
    const size_t most = 227 * 1024 - 1024;
    int nb = 1, cl = 1, nt = 256;
    auto seg = [&](int blocks) { return (units + blocks - 1) / blocks * unit * (long long)sizeof(T); };   // bytes of a row
    auto piece = [&] { return (double)((a.pixels + cl - 1) / cl) * seg(nb); };
    for (;;) {
        const bool few = (long long)a.n * nb * cl < 2 * sms;
        if (!few && piece() <= 72 * 1024) break;
        if (nb < units && seg(2 * nb) >= 128) nb *= 2;
        else if (cl < (few ? 16 : 8) && a.pixels >= 16 * cl && piece() > 16 * 1024) cl *= 2;
        else if (few && nb < units && seg(2 * nb) >= 32) nb *= 2;
        else break;
    }
    const int per = (units + nb - 1) / nb;
    a.cb = (int)(per * unit), a.nb = (units + per - 1) / per;
    a.ppc = (a.pixels + cl - 1) / cl;
    if ((long long)a.n * a.nb * cl <= sms) nt = 512;
    const size_t fixed = maps_fixed<V>(nt, a.cb / a.cpg), row = (size_t)a.cb * sizeof(T);
    if (fixed > most) return cudaErrorInvalidConfiguration;
    a.hold = (int)(a.ppc < (long long)((most - fixed) / row) ? a.ppc : (long long)((most - fixed) / row));
    const size_t smem = fixed + a.hold * row;
    static std::atomic<unsigned long long> attr{0};
    const unsigned long long ctx = fcm_current_ctx_id();
    if (ctx == 0 || attr.load(std::memory_order_relaxed) != ctx) {
        cudaError_t e = cudaFuncSetAttribute(norm_maps_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(norm_maps_kernel<T, V>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        attr.store(ctx, std::memory_order_relaxed);
    }
    return launch(norm_maps_kernel<T, V>, dim3((unsigned)((long long)a.n * a.nb * cl)), nt, smem, st, a, cl);
}

template <typename T, int V, int LPG, int NV, int ROWS> static cudaError_t rows_kernel(const NormArgs &a, cudaStream_t st) {
    const long long units = (long long)(a.n + ROWS - 1) / ROWS * a.groups;
    return launch(norm_rows_kernel<T, V, LPG, NV, ROWS>, dim3((unsigned)((units * LPG + 255) / 256)), 256, 0, st, a);
}

template <typename T> static cudaError_t run_norm(const NormArgs &a, int sms, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = aligned16(a.x) && aligned16(a.y) && aligned16(a.z) &&
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
    return vec ? run_maps<T, V>(a, sms, st) : run_maps<T, 1>(a, sms, st);
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
