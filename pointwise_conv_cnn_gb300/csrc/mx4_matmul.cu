// mx4_matmul.cu -- pointwise layer whose rows and weights are both microscaled 4-bit.
//
//     y[t,o] = act(s[o] * sum_i x[t,i] * w[o,i] + b[o])
#include <atomic>

#include "mx4.cuh"
#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct Mx4MatmulArgs {
    CUtensorMap wmap, xmap;   // rows of bytes: weights, tokens
    const uint8_t *ws, *xs;
    const float *s, *b;
    void *y;
    long long ld_y;
    int m, out, groups, act, dtype;
    int chunks;        // of 512 inputs
    int split;         // blocks of a cluster, which share the inputs
    int wvec, xvec;    // rows of scales may be read 16 bytes at a time
};

// Descriptor of a product of microscaled 4-bit factors (E2M1, scales powers of two): 128 x n x 64, both factors with
// their inputs side by side; `sf` selects bytes sf, sf + 1 of each scale word.
__host__ __device__ constexpr uint32_t idesc_mx4(int n, uint32_t sf) {
    return sf << 4 | 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | 1u << 23 | 1u << 27 | sf << 29;
}
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 32 rows of 16 bytes, side by side in shared memory, to four columns of each of the tensor memory's quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
    const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1 << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// A block: 128 outputs of NT tokens.  Rows of the product are outputs, so that a warp's stores of a token are side by
// side.  Inputs go in stages of 256, 128 bytes a row.  Two blocks share an SM, so that one's end (its sums' way out, about
// a quarter of its products' time at 8192 inputs) lies under the other's products: one block of 256 tokens, whose products
// need less of shared memory's bandwidth, took 161 us for 4096 x 8192 x 8192 where these take 147.
template <int NT> struct Mx4Shape {
    static constexpr int ST = NT == 128 ? 3 : 4;             // stages
    static constexpr int A = 128 * 128, B = NT * 128;        // bytes of a stage
    static constexpr int SF = 1024;                          // of each factor's scales: two words of four for each row
    static constexpr int SMEM = ST * (A + B + 2 * SF) + 1024 /* alignment */ + 256 /* barriers */;
    static constexpr int ACC = NT < 32 ? 32 : NT;
    static constexpr int SFC = 16;                           // columns of a stage's scales
    static constexpr int COLS = ACC + ST * SFC <= 128 ? 128 : 256;
    static_assert(ST * (A + B) >= 128 * NT * 4, "the sums of a split product take the stages' place");
    static_assert(2 * (SMEM + 1024) <= 228 * 1024 && ACC + ST * SFC <= COLS, "two blocks an SM");
};

// The 16 scale codes of `rows` rows for one chunk of 512 inputs, by a warp: on their way to shared memory as 4 blocks
// (of 128 inputs) of 32 x 16 bytes, row r's word at (r % 32) * 16 + (r / 32) * 4.  Where rows of codes start at 16
// bytes a lane has rows lane, lane + 32, .. whole, and stores 16 bytes a block.  Else four lanes have a row, a word
// each, taken from the two aligned words that it lies in, which are put together only when they are stored: the
// loads of the next chunk are under way meanwhile.
struct ScaleChunk {
    uint32_t lo[16], hi[16];
    uint32_t shift, keep;
    __device__ __forceinline__ void load(const uint8_t *s, int vec, int row0, int rows, int last_row, int groups, int g0, int lane) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (i * 32 < rows) v = *reinterpret_cast<const uint4 *>(s + (size_t)min(row0 + i * 32 + lane, last_row) * groups + g0);
                lo[i * 4] = v.x, lo[i * 4 + 1] = v.y, lo[i * 4 + 2] = v.z, lo[i * 4 + 3] = v.w;
            }
        } else {
            const int g = g0 + lane % 4 * 4, have = min(groups - g, 4);   // codes of this word
            // rows 8 apart lie alike in their words; one past the last row is that row, and comes out as anything
            shift = (uint32_t)(reinterpret_cast<uintptr_t>(s) + (size_t)(row0 + lane / 4) * groups + g) % 4 * 8;
            keep = have >= 4 ? ~0u : have <= 0 ? 0u : (1u << (8 * have)) - 1;   // codes past the last: any number
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const uintptr_t at = reinterpret_cast<uintptr_t>(s + (size_t)min(row0 + i * 8 + lane / 4, last_row) * groups + g);
                const int off = (int)(at & 3);
                const uint32_t *p = reinterpret_cast<const uint32_t *>(at - off);
                lo[i] = hi[i] = 0;
                if (i * 8 < rows && have > 0) lo[i] = p[0];
                if (i * 8 < rows && off + have > 4) hi[i] = p[1];
            }
        }
    }
    // the blocks 2 * half and 2 * half + 1, one stage's
    __device__ __forceinline__ void store(uint32_t to, int vec, int half, int lane) const {
        if (vec) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                if (half == 0) tc::sts128(to + k * 512 + lane * 16, lo[k], lo[4 + k], lo[8 + k], lo[12 + k]);
                else tc::sts128(to + k * 512 + lane * 16, lo[2 + k], lo[6 + k], lo[10 + k], lo[14 + k]);
            }
        } else if ((lane & 2) == 2 * half) {
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int r = i * 8 + lane / 4;
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + (lane & 1) * 512 + r % 32 * 16 + r / 32 * 4),
                             "r"(__funnelshift_r(lo[i], hi[i], shift) & keep) : "memory");
            }
        }
    }
};

__device__ __forceinline__ void mx4_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// N tokens' sums of output o as results.
template <int N> __device__ __forceinline__ void mx4_values(const Mx4MatmulArgs &a, int o, float (&v)[N]) {
    const float f = a.s ? a.s[o] : 1.0f, b = a.b ? a.b[o] : 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = fmaf(f, v[i], b);
    if (a.act == FCM_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = silu(v[i]);
    } else if (a.act != FCM_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = clamp_act(v[i], a.act);
    }
}

// A lane's output of the block's tokens, from tensor memory; a warp's stores of a token are side by side.
template <typename T, int NT>
__device__ __forceinline__ void mx4_finish(const Mx4MatmulArgs &a, uint32_t acc, int o, int m0, bool ok) {
    T *y = static_cast<T *>(a.y) + (long long)m0 * a.ld_y + o;
    const bool mine = o < a.out;
    const int last = min(o, a.out - 1);
    for (int c = 0; c < NT && m0 + c < a.m; c += 16) {
        uint32_t r[16];
        float v[16];
        tc::tmem_ld16(acc + c, r);
        tc::tmem_ld_wait(r, r);
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = __uint_as_float(ok ? r[i] : 0x7FFFFFFFu);
        mx4_values<16>(a, last, v);
        const int n = mine ? a.m - m0 - c : 0;
        if (n >= 16) {
#pragma unroll
            for (int i = 0; i < 16; i++) y[(c + i) * a.ld_y] = Storage<T>::from_f(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; i++)
                if (i < n) y[(c + i) * a.ld_y] = Storage<T>::from_f(v[i]);
        }
        __syncwarp();
    }
}

template <typename T>
__device__ __forceinline__ void mx4_put(const Mx4MatmulArgs &a, int t, int o, int n, const float (&v)[8]) {
    T *y = static_cast<T *>(a.y) + (long long)t * a.ld_y + o;
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (i < n) y[i * a.ld_y] = Storage<T>::from_f(v[i]);
}

// Warp 0 asks for the factors (TMA), warp 1 multiplies, warps 4 and 5 bring the scales to shared memory, from where warp
// 1 has them copied to tensor memory ahead of its products, and warps 4 to 7 finish.  A bounded wait that runs out ends
// the block with NaN for its outputs.
//
// 4096 x 8192 x 8192: 146 us, 3.76 PFLOP/s, twice the 16-bit rate of the library's product.  What binds is shared memory,
// which takes 8 KB in and gives 8 KB out for a product of 128 x 128 x 64, 128 cycles at 128 bytes, where the product itself
// takes 64 (the tensor cores are 41 % busy): pairs of SMs on one tile would halve the tokens' share.  16 tokens through
// 20480 x 8192: 89 MB of weights and scales in 18.9 us, 4.8 TB/s, 0.70 of a plain copy's rate.
template <int NT> __global__ void __launch_bounds__(256, 2) mx4_matmul_kernel(const __grid_constant__ Mx4MatmulArgs a) {
    using S = Mx4Shape<NT>;
    extern __shared__ unsigned char raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ unsigned error;
    const uint32_t base = (tc::smem_u32(raw) + 1023) & ~1023u;
    const uint32_t at_a = base, at_b = at_a + S::ST * S::A, at_sf = at_b + S::ST * S::B, bars = at_sf + S::ST * 2 * S::SF;
    const uint32_t full = bars, sf_full = bars + 8 * S::ST, empty = bars + 16 * S::ST, done = bars + 24 * S::ST;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const unsigned tile = blockIdx.x / a.split, rank = blockIdx.x % a.split, tiles_m = ((unsigned)a.m + NT - 1) / NT;
    const int m0 = (int)(tile % tiles_m) * NT, o0 = (int)(tile / tiles_m) * 128;
    const int c0 = (int)((long long)a.chunks * rank / a.split), c1 = (int)((long long)a.chunks * (rank + 1) / a.split);
    const int stages = min(2 * c1, (a.groups + 7) / 8) - 2 * c0;   // of 8 codes
    volatile int *abort = &abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0, error = 0;
        for (int i = 0; i < S::ST; i++) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(sf_full + 8 * i, 2);
            tc::mbar_init(empty + 8 * i, 1);
        }
        tc::mbar_init(done, 1);
        tc::fence_barrier_init();
        tc::tma_prefetch_desc(&a.wmap);
        tc::tma_prefetch_desc(&a.xmap);
    }
    if (warp == 2) tc::tmem_alloc(tc::smem_u32(&tmem_slot), S::COLS);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    auto wait = [&](uint32_t bar, uint32_t parity) { return tc::mbar_wait(bar, parity, abort, &error, tc::kWaitLimitNs); };

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (; it < stages; it++) {
                const int s = it % S::ST;
                if (it >= S::ST && !wait(empty + 8 * s, (it / S::ST - 1) & 1)) break;
                tc::mbar_arrive_expect_tx(full + 8 * s, S::A + S::B);
                const int x = (2 * c0 + it) * 128;
                tc::tma_load_2d(at_a + s * S::A, &a.wmap, full + 8 * s, x, o0);
                tc::tma_load_2d(at_b + s * S::B, &a.xmap, full + 8 * s, x, m0);
            }
            // what is on its way has arrived before the block ends
            for (int i = max(0, it - S::ST); i < it; i++)
                for (int n = 0; n < (1 << 20) && !tc::mbar_try_wait(full + 8 * (i % S::ST), (i / S::ST) & 1); n++) {}
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t sft = tmem + S::ACC;
            for (int it = 0; it < stages; it++) {
                const int s = it % S::ST;
                const uint32_t phase = (it / S::ST) & 1;
                if (!wait(full + 8 * s, phase) || !wait(sf_full + 8 * s, phase)) break;
                tc::tc_fence_after();
                const uint32_t sf = at_sf + s * 2 * S::SF, sfa = sft + s * S::SFC, sfb = sfa + 8;
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    copy_scales(sfa + k * 4, sf + k * 512);
                    copy_scales(sfb + k * 4, sf + S::SF + k * 512);
                }
                const uint64_t ad = tc::sw128_kmajor_desc(at_a + s * S::A), bd = tc::sw128_kmajor_desc(at_b + s * S::B);
#pragma unroll
                for (int j = 0; j < 4; j++)
                    mma_mx4(tmem, tc::desc_advance(ad, j * 32), tc::desc_advance(bd, j * 32), idesc_mx4(NT, (j & 1) * 2),
                            sfa + j / 2 * 4, sfb + j / 2 * 4, (it | j) != 0);
                tc::mma_commit(empty + 8 * s);
            }
            tc::mma_commit(done);
        }
    } else if (warp >= 4) {
        const int role = warp - 4;   // 0: weights' scales, 1: tokens'
        if (role < 2) {
            const uint8_t *src = role ? a.xs : a.ws;
            const int vec = role ? a.xvec : a.wvec, row0 = role ? m0 : o0;
            const int last = (role ? a.m : a.out) - 1, rows = role ? NT : 128;
            ScaleChunk chunk[2];
            bool ok = true;
            auto stage_pair = [&](const ScaleChunk &now, int it) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (it + h >= stages || !ok) break;
                    const int s = (it + h) % S::ST;
                    if (it + h >= S::ST) ok = wait(empty + 8 * s, ((it + h) / S::ST - 1) & 1);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    now.store(at_sf + (2 * s + role) * S::SF, vec, h, lane);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(sf_full + 8 * s);
                }
            };
            auto load = [&](ScaleChunk &to, int it) {
                if (it < stages) to.load(src, vec, row0, rows, last, a.groups, (2 * c0 + it) * 8, lane);
            };
            load(chunk[0], 0);
            for (int it = 0; it < stages && ok; it += 4) {
                load(chunk[1], it + 2);
                stage_pair(chunk[0], it);
                load(chunk[0], it + 4);
                stage_pair(chunk[1], it + 2);
            }
        }
        // the sums: a lane has an output, a column is a token's
        const bool ok = __all_sync(~0u, wait(done, 0)) && !*abort;
        tc::tc_fence_after();
        const uint32_t acc = tmem + ((uint32_t)role << 21);   // the warp's quarter of the lanes
        if (a.split == 1) {
            if (a.dtype == FCM_BF16) mx4_finish<__nv_bfloat16, NT>(a, acc, o0 + role * 32 + lane, m0, ok);
            else if (a.dtype == FCM_F16) mx4_finish<__half, NT>(a, acc, o0 + role * 32 + lane, m0, ok);
            else mx4_finish<float, NT>(a, acc, o0 + role * 32 + lane, m0, ok);
        } else {
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                tc::tmem_ld16(acc + c, r);
                tc::tmem_ld_wait(r, r);
#pragma unroll
                for (int i = 0; i < 16; i++)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + ((c + i) * 128 + role * 32 + lane) * 4),
                                 "r"(ok ? r[i] : 0x7FFFFFFFu) : "memory");
            }
        }
        tc::tc_fence_before();
        if (a.split > 1) {
            __syncwarp();
            mx4_cluster_sync();
            // each block of the cluster joins its share of the tokens, in the blocks' order
            const int n0 = NT * (int)rank / a.split, n1 = NT * (int)(rank + 1) / a.split;
            const int o = o0 + role * 32 + lane;
            for (int c = n0; c < n1 && m0 + c < a.m; c += 8) {
                float v[8] = {};
                for (int r = 0; r < a.split; r++) {
                    uint32_t addr;
                    float p[8];
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(base + (c * 128 + role * 32 + lane) * 4), "r"(r));
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p[i]) : "r"(addr + min(i, n1 - 1 - c) * 512) : "memory");
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] += p[i];
                }
                if (o < a.out) {
                    const int n = min(n1 - c, a.m - m0 - c);
                    mx4_values<8>(a, o, v);
                    if (a.dtype == FCM_BF16) mx4_put<__nv_bfloat16>(a, m0 + c, o, n, v);
                    else if (a.dtype == FCM_F16) mx4_put<__half>(a, m0 + c, o, n, v);
                    else mx4_put<float>(a, m0 + c, o, n, v);
                }
            }
        }
    }
    if (a.split > 1) {
        __syncwarp();
        if (warp < 4) mx4_cluster_sync();
        mx4_cluster_sync();   // the others may still read this block's sums
    }
    __syncthreads();
    if (warp == 2) tc::tmem_dealloc(tmem, S::COLS);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// Rows of `bytes` bytes, `box` rows of 128 bytes at a time, 128-byte swizzled; what is past the end comes as zeros.
static bool byte_map(CUtensorMap *map, const void *p, long long bytes, long long rows, int box) {
    const cuuint64_t dim[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)bytes};
    const cuuint32_t size[2] = {128, (cuuint32_t)box}, step[2] = {1, 1};
    const EncodeTiled enc = encode_tiled();
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dim, stride, size, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
static cudaError_t run_mx4(Mx4MatmulArgs &a, const void *wq, const void *xq, int sms, cudaStream_t st) {
    using S = Mx4Shape<NT>;
    const long long bytes = a.groups * 16ll;
    if (!byte_map(&a.wmap, wq, bytes, a.out, 128) || !byte_map(&a.xmap, xq, bytes, a.m, NT)) return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> attr{0};
    const unsigned long long ctx = fcm_current_ctx_id();
    if (ctx == 0 || attr.load(std::memory_order_relaxed) != ctx) {
        const cudaError_t e = cudaFuncSetAttribute(mx4_matmul_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        attr.store(ctx, std::memory_order_relaxed);
    }
    const long long tiles = ((a.m + NT - 1ll) / NT) * ((a.out + 127ll) / 128);
    // Blocks that share the inputs of a tile, where the tiles leave SMs without a block.  More than four, and for 128
    // tokens a second block an SM, cost more than they bring.  Measured, us without sharing, with two, four and eight: 16
    // tokens, 4096 x 4096 (32 tiles) 9.2, -, 6.5, 8.4; 300 tokens, 1000 x 8192 (24) 19.7, -, 11.8, 12.7; 16 tokens, 8192 x
    // 8192 (64) 16.2, 11.5, 10.8; 256 tokens, 8192 x 4096 (128) 12.1, 14.2; 333 tokens, 5003 x 4128 (120) 15.8, 18.0.
    const long long most = (long long)sms * (NT < 128 ? 2 : 1);
    a.split = 1;
    while (a.split < 4 && tiles * a.split * 2 <= most && 2 * a.split <= a.chunks) a.split *= 2;
    return launch(mx4_matmul_kernel<NT>, dim3((unsigned)(tiles * a.split)), 256, S::SMEM, st, a, a.split);
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
    const long long most = ((d.m + 15ll) / 16) * ((d.out + 127ll) / 128);   // blocks of the smallest tiles
    if (most * 8 > 0x7FFFFFFFLL) return fcm_fail(FCM_ERR_UNSUPPORTED, "m %d, out %d: above 2^31 - 1 blocks", d.m, d.out);
    seq::Mx4MatmulArgs a = {};
    a.ws = static_cast<const uint8_t *>(ws), a.xs = static_cast<const uint8_t *>(xs), a.s = s, a.b = b, a.y = y;
    a.ld_y = d.ld_y, a.m = d.m, a.out = d.out, a.groups = (int)groups, a.act = d.act, a.dtype = d.dtype;
    a.chunks = (int)((groups + 15) / 16);
    a.wvec = seq::aligned16(ws) && groups % 16 == 0, a.xvec = seq::aligned16(xs) && groups % 16 == 0;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t ce = d.m <= 16   ? seq::run_mx4<16>(a, wq, xq, sms, cs)
                           : d.m <= 32 ? seq::run_mx4<32>(a, wq, xq, sms, cs)
                           : d.m <= 64 ? seq::run_mx4<64>(a, wq, xq, sms, cs)
                                       : seq::run_mx4<128>(a, wq, xq, sms, cs);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
