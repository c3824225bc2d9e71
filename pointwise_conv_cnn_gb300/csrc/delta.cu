// delta.cu -- the gated delta rule: argument checks, the choice of kernel, and the kernel that goes row by
// row.
//
//     S = e^G S;  u = B (v - S^T k);  S = S + k u^T;  y = scale S^T q
#include <atomic>

#include "delta_chunk.cuh"

namespace fcm {
namespace seq {

// Row by row.  A block has 32 of a head's value columns, a thread four of them and every 16th row of the state, in
// registers.  Both products with the state need its value before the row only,
//     u = B (v - e^G S^T k),   S^T q after it = e^G S^T q + (q.k) u,
// so that a row costs one sum over 16 threads.  Rows come in batches: their norms, products q.k, decays
// and steps are made once for all columns by a warp a row.  VEC: four columns of the state, v and y are read and
// written at once.
// LONG (prompts): the 16 threads are a warp's, so that no row waits at a barrier, and the next batch is on its
// way while one is computed.  For single tokens they are a block's, whose warps then read and write the state's rows in
// pieces of 128 bytes instead of 32 (128 sequences of 32 heads 95 us, 113 as for prompts), with registers for six
// blocks an SM.
//
// Single tokens are bound by their states' way in and out: 128 sequences of 32 heads of 128 x 128 move 540 MB in 95 us, 5.7
// TB/s, 0.84 of a plain copy's rate; one sequence of 16 heads takes 3.6 us, a launch and a chain of loads.  Prompts in
// 32 bits, and what the chunks do not take, cost the latency of a row's sums: 777 x 8 heads of 128 x 128 317 us.
template <typename T, int RK, bool VEC, bool LONG>
__global__ void __launch_bounds__(128, LONG ? 3 : RK <= 8 ? 6 : 3) delta_row_kernel(const DeltaArgs a) {
    constexpr int TB = 8, DK = 16 * RK, DV = kDeltaCols, KN = TB * DK / 128, VN = TB * DV / 128;
    __shared__ float qs[TB][DK], ks[TB][DK], vs[TB][DV];
    __shared__ float4 row[TB];    // e^G, B, 1 / |k|, scale / |q|
    __shared__ float prod[TB];    // q.k
    __shared__ float4 red[LONG ? 1 : 2][4][8][2];
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, tx = LONG ? 2 * warp + lane % 2 : threadIdx.x % 8,
              ty = LONG ? lane / 2 : threadIdx.x / 8;
    const int slice = blockIdx.x % a.slices, rest = blockIdx.x / a.slices;
    const int h = rest % a.heads, q = rest / a.heads, g = h / a.per_key;
    long long t0;
    int len;
    seq_rows(a.q, q, t0, len);
    const int at = a.state_in || a.state_out ? state_row(a.q, q) : -1;
    const int d0 = slice * DV, d = d0 + 4 * tx;
    const size_t cell = ((size_t)max(at, 0) * a.heads + h) * a.dk * a.dv + d;
    float s[RK][4];
    const bool from = a.state_in && at >= 0;
#pragma unroll
    for (int r = 0; r < RK; r++) {
        const int i = ty + 16 * r;
        const float *p = a.state_in + cell + (size_t)i * a.dv;
        if (VEC) {
            const float4 v = from && i < a.dk && d < a.dv ? *reinterpret_cast<const float4 *>(p) : make_float4(0, 0, 0, 0);
            s[r][0] = v.x, s[r][1] = v.y, s[r][2] = v.z, s[r][3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) s[r][e] = from && i < a.dk && d + e < a.dv ? p[e] : 0.0f;
        }
    }
    const T *qp = static_cast<const T *>(a.qp) + (size_t)g * a.dk, *kp = static_cast<const T *>(a.kp) + (size_t)g * a.dk;
    const T *vp = static_cast<const T *>(a.vp) + (size_t)h * a.dv + d0;
    T *y = static_cast<T *>(a.y) + (size_t)h * a.dv + d;
    const float av = a.a[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    // element i of a batch's keys, queries (row i / DK) or values (i / DV), zeros past the rows and columns
    auto element = [&](const T *p, long long ld, int b0, int i, int width, int columns) {
        const int j = i / width, e = i % width;
        return b0 + j < len && e < columns ? p[(t0 + b0 + j) * ld + e] : Storage<T>::from_f(0.0f);
    };
    T kn[LONG ? KN : 1], qn[LONG ? KN : 1], vn[LONG ? VN : 1], dtn[2], bn[2];
    auto scalars = [&](int b0) {   // of this warp's rows: warp, warp + 4
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const bool live = b0 + warp + 4 * i < len;
            const long long t = live ? t0 + b0 + warp + 4 * i : t0;
            dtn[i] = live ? static_cast<const T *>(a.dt)[t * a.ld_dt + h] : Storage<T>::from_f(0.0f);
            bn[i] = live ? static_cast<const T *>(a.b)[t * a.ld_b + h] : Storage<T>::from_f(0.0f);
        }
    };
    auto fetch = [&](int b0) {
#pragma unroll
        for (int i = 0; i < KN; i++) {
            kn[i] = element(kp, a.ld_k, b0, threadIdx.x + 128 * i, DK, a.dk);
            qn[i] = element(qp, a.ld_q, b0, threadIdx.x + 128 * i, DK, a.dk);
        }
#pragma unroll
        for (int i = 0; i < VN; i++) vn[i] = element(vp, a.ld_v, b0, threadIdx.x + 128 * i, DV, a.dv - d0);
    };
    if (len > 0) {
        scalars(0);
        if constexpr (LONG) fetch(0);
    }
    for (int b0 = 0, n; b0 < len; b0 += n) {
        n = min(TB, len - b0);
        if constexpr (LONG) {
#pragma unroll
            for (int i = 0; i < KN; i++) {
                (&ks[0][0])[threadIdx.x + 128 * i] = Storage<T>::to_f(kn[i]);
                (&qs[0][0])[threadIdx.x + 128 * i] = Storage<T>::to_f(qn[i]);
            }
#pragma unroll
            for (int i = 0; i < VN; i++) (&vs[0][0])[threadIdx.x + 128 * i] = Storage<T>::to_f(vn[i]);
        } else {
            for (int i = threadIdx.x; i < n * DK; i += 128) {
                (&ks[0][0])[i] = Storage<T>::to_f(element(kp, a.ld_k, b0, i, DK, a.dk));
                (&qs[0][0])[i] = Storage<T>::to_f(element(qp, a.ld_q, b0, i, DK, a.dk));
            }
            for (int i = threadIdx.x; i < n * DV; i += 128) (&vs[0][0])[i] = Storage<T>::to_f(element(vp, a.ld_v, b0, i, DV, a.dv - d0));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int j = warp + 4 * i;
            if (j >= n) break;
            float qq = 0.0f, kk = 0.0f, qk = 0.0f;
#pragma unroll
            for (int e = lane; e < DK; e += 32) {
                const float x = qs[j][e], z = ks[j][e];
                qq = fmaf(x, x, qq), kk = fmaf(z, z, kk), qk = fmaf(x, z, qk);
            }
#pragma unroll
            for (int m = 16; m; m >>= 1) {
                qq += __shfl_xor_sync(~0u, qq, m), kk += __shfl_xor_sync(~0u, kk, m), qk += __shfl_xor_sync(~0u, qk, m);
            }
            if (lane == 0) {
                row[j] = make_float4(expf(log_decay(Storage<T>::to_f(dtn[i]) + bias, av, a.softplus)),
                                     step_of(Storage<T>::to_f(bn[i]), a.sigmoid), a.normalize ? rsqrtf(kk + kDeltaEps) : 1.0f,
                                     a.normalize ? a.scale * rsqrtf(qq + kDeltaEps) : a.scale);
                prod[j] = qk;
            }
        }
        __syncthreads();
        if (len - b0 > TB) {
            scalars(b0 + TB);
            if constexpr (LONG) fetch(b0 + TB);
        }
        for (int j = 0; j < n; j++) {
            float pk[4] = {}, pq[4] = {}, kr[RK];
#pragma unroll
            for (int r = 0; r < RK; r++) {
                kr[r] = ks[j][ty + 16 * r];
                const float qr = qs[j][ty + 16 * r];
#pragma unroll
                for (int e = 0; e < 4; e++) pk[e] = fmaf(kr[r], s[r][e], pk[e]), pq[e] = fmaf(qr, s[r][e], pq[e]);
            }
#pragma unroll
            for (int m = LONG ? 2 : 8; m < 32; m <<= 1)
#pragma unroll
                for (int e = 0; e < 4; e++) pk[e] += __shfl_xor_sync(~0u, pk[e], m), pq[e] += __shfl_xor_sync(~0u, pq[e], m);
            if constexpr (!LONG) {
                auto &sums = red[j & 1];
                if (lane < 8) {
                    sums[warp][tx][0] = make_float4(pk[0], pk[1], pk[2], pk[3]);
                    sums[warp][tx][1] = make_float4(pq[0], pq[1], pq[2], pq[3]);
                }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 4; e++) pk[e] = pq[e] = 0.0f;
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const float4 x = sums[w][tx][0], z = sums[w][tx][1];
                    pk[0] += x.x, pk[1] += x.y, pk[2] += x.z, pk[3] += x.w;
                    pq[0] += z.x, pq[1] += z.y, pq[2] += z.z, pq[3] += z.w;
                }
            }
            const float4 f = row[j], v = *reinterpret_cast<const float4 *>(&vs[j][4 * tx]);
            const float fk = f.x * f.z;
            const float u[4] = {f.y * fmaf(-fk, pk[0], v.x), f.y * fmaf(-fk, pk[1], v.y), f.y * fmaf(-fk, pk[2], v.z),
                                f.y * fmaf(-fk, pk[3], v.w)};
#pragma unroll
            for (int r = 0; r < RK; r++) {
                const float k = f.z * kr[r];
#pragma unroll
                for (int e = 0; e < 4; e++) s[r][e] = fmaf(k, u[e], f.x * s[r][e]);
            }
            if (ty == 0) {
                const float qk = f.z * prod[j];
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; e++) o[e] = f.w * fmaf(qk, u[e], f.x * pq[e]);
                T *to = y + (t0 + b0 + j) * a.ld_y;
                if (VEC) {
                    if (d < a.dv) {
                        Vec<T, 4> v4;
                        v4.put(o);
                        *reinterpret_cast<Vec<T, 4> *>(to) = v4;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (d + e < a.dv) to[e] = Storage<T>::from_f(o[e]);
                }
            }
        }
        __syncthreads();   // the next batch overwrites this one's rows
    }
    if (a.state_out && at >= 0) {
#pragma unroll
        for (int r = 0; r < RK; r++) {
            const int i = ty + 16 * r;
            float *p = a.state_out + cell + (size_t)i * a.dv;
            if (i >= a.dk) continue;
            if (VEC) {
                if (d < a.dv) *reinterpret_cast<float4 *>(p) = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (d + e < a.dv) p[e] = s[r][e];
            }
        }
    }
}

// Longest sequence's rows from which prompts go in chunks.  Where blocks are few chunks are ahead from 10 rows or so on, where
// they are many from 18; the rule asks for neither, nor how many sequences are as long as the longest.  Measured, us, heads of 128 x
// 128, bf16, states in the L2: 1 sequence of 32 heads, 4, 8, 12, 15 rows 4.1, 5.6, 7.5, 8.7 row by row, 16 rows 6.5 in chunks; 64 of
// 8 heads, 4, 8, 12, 15 rows 26, 37, 52, 61, 16 rows 69 in chunks.  A single token in a batch that goes in chunks costs a chunk's
// time and an SM of its own: 127 of 32 heads and a prompt of 512 rows 560 us together, 99 and 38 as two calls; 128 with a loose
// bound of their lengths 530, with a bound of 1 100.
constexpr int kChunkedFrom = 16;
// ... and from which the row kernel is the prompts': 64 sequences of 8 heads, 2, 4, 8 rows 21.4, 27.0, 40.2 us, as single
// tokens 20.3, 28.2, 44.7.
constexpr int kManyFrom = 3;

template <typename T, int DK> static cudaError_t run_chunks(const DeltaArgs &a, dim3 grid, cudaStream_t st) {
    static std::atomic<unsigned long long> attr{0};
    const unsigned long long ctx = fcm_current_ctx_id();
    if (ctx == 0 || attr.load(std::memory_order_relaxed) != ctx) {
        const cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<T, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   DeltaChunk<DK>::SMEM);
        if (e != cudaSuccess) return e;
        attr.store(ctx, std::memory_order_relaxed);
    }
    return launch(delta_chunk_kernel<T, DK>, grid, DeltaChunk<DK>::THREADS, DeltaChunk<DK>::SMEM, st, a);
}

template <typename T> static cudaError_t run_delta(DeltaArgs a, cudaStream_t st) {
    const size_t v = 4 * sizeof(T);
    auto by = [](const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const bool vec = a.dv % 4 == 0 && by(a.state_in, 16) && by(a.state_out, 16) && by(a.y, v) && a.ld_y % 4 == 0;
    const dim3 grid((unsigned)((long long)a.q.n_seq * a.heads * a.slices));
    if constexpr (sizeof(T) == 2) {
        a.vec = by(a.qp, 16) && by(a.kp, 16) && ((a.ld_q | a.ld_k | a.dk) % 8) == 0;
        a.vec_v = by(a.vp, 16) && ((a.ld_v | a.dv) % 8) == 0;
        if (a.q.max_len >= kChunkedFrom && a.dk <= 128)
            return a.dk <= 64 ? run_chunks<T, 64>(a, grid, st) : run_chunks<T, 128>(a, grid, st);
    }
    auto rows = [&](void (*one)(DeltaArgs), void (*one_vec)(DeltaArgs), void (*many)(DeltaArgs), void (*many_vec)(DeltaArgs)) {
        return launch(a.q.max_len >= kManyFrom ? (vec ? many_vec : many) : (vec ? one_vec : one), grid, 128, 0, st, a);
    };
#define ROWS(rk) \
    rows(delta_row_kernel<T, rk, false, false>, delta_row_kernel<T, rk, true, false>, delta_row_kernel<T, rk, false, true>, \
         delta_row_kernel<T, rk, true, true>)
    return a.dk <= 64 ? ROWS(4) : a.dk <= 128 ? ROWS(8) : ROWS(16);
#undef ROWS
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_gated_delta(const fcm_delta_desc *desc, const void *q, const void *k, const void *v,
                                      const void *dt, const float *a, const void *b, const float *dt_bias,
                                      const float *state_in, void *y, float *state_out, void *stream) {
    FcmNvtxRange nvtx("fcm_gated_delta");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_delta_desc d = *desc;
    if (d.heads < 1 || d.key_heads < 1 || d.dk < 1 || d.dv < 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "heads %d, key_heads %d, dk %d, dv %d", d.heads, d.key_heads, d.dk, d.dv);
    if (d.heads % d.key_heads)
        return fcm_fail(FCM_ERR_INVALID_ARG, "%d key heads do not divide %d heads", d.key_heads, d.heads);
    if (d.dk > seq::kMaxDeltaKeys) return fcm_fail(FCM_ERR_UNSUPPORTED, "dk %d above %d", d.dk, seq::kMaxDeltaKeys);
    if (d.dtype < FCM_F32 || d.dtype > FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d.dtype);
    for (const int flag : {d.softplus, d.sigmoid, d.normalize})
        if (flag != 0 && flag != 1)
            return fcm_fail(FCM_ERR_INVALID_ARG, "softplus %d, sigmoid %d, normalize %d: 0 or 1", d.softplus, d.sigmoid,
                            d.normalize);
    const long long ck = (long long)d.key_heads * d.dk, cv = (long long)d.heads * d.dv;
    if (cv * d.dk > 0x7FFFFFFFLL) return fcm_fail(FCM_ERR_UNSUPPORTED, "heads * dk * dv above 2^31 - 1");
    seq::DeltaArgs g = {};
    fcm_status st;
    if ((st = seq::check_seqs(d.seqs, state_in || state_out, &g.q)) != FCM_OK ||
        (st = seq::check_ld(&d.ld_q, ck, "ld_q")) != FCM_OK || (st = seq::check_ld(&d.ld_k, ck, "ld_k")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_v, cv, "ld_v")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_dt, d.heads, "ld_dt")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_b, d.heads, "ld_b")) != FCM_OK || (st = seq::check_ld(&d.ld_y, cv, "ld_y")) != FCM_OK)
        return st;
    if (g.q.n_seq == 0) return FCM_OK;
    const size_t e = (size_t)fcm_dtype_bytes(d.dtype);
    const long long rows = g.q.tokens;   // without rows the activations may be NULL
    if ((rows && ((st = seq::check_dev_ptr(q, e, "q")) != FCM_OK || (st = seq::check_dev_ptr(k, e, "k")) != FCM_OK ||
                  (st = seq::check_dev_ptr(v, e, "v")) != FCM_OK || (st = seq::check_dev_ptr(dt, e, "dt")) != FCM_OK ||
                  (st = seq::check_dev_ptr(b, e, "b")) != FCM_OK || (st = seq::check_dev_ptr(y, e, "y")) != FCM_OK)) ||
        (st = seq::check_dev_ptr(a, 4, "a")) != FCM_OK ||
        (dt_bias && (st = seq::check_dev_ptr(dt_bias, 4, "dt_bias")) != FCM_OK) ||
        (state_in && (st = seq::check_dev_ptr(state_in, 4, "state_in")) != FCM_OK) ||
        (state_out && (st = seq::check_dev_ptr(state_out, 4, "state_out")) != FCM_OK))
        return st;
    const struct {
        const void *p;
        long long ld, cols;
        const char *name;
    } ins[] = {{q, d.ld_q, ck, "q"}, {k, d.ld_k, ck, "k"}, {v, d.ld_v, cv, "v"}, {dt, d.ld_dt, d.heads, "dt"},
               {b, d.ld_b, d.heads, "b"}};
    for (const auto &in : ins)
        if (seq::rows_overlap(in.p, in.ld, in.cols, y, d.ld_y, cv, rows, e))
            return fcm_fail(FCM_ERR_INVALID_ARG, "%s and y overlap", in.name);
    const long long cells = cv * d.dk;
    if (state_in != state_out && seq::rows_overlap(state_in, cells, cells, state_out, cells, cells, g.q.slots, 4))
        return fcm_fail(FCM_ERR_INVALID_ARG, "state_in and state_out overlap without being the same");
    g.slices = (d.dv + seq::kDeltaCols - 1) / seq::kDeltaCols;
    if ((long long)g.q.n_seq * d.heads * g.slices > 0x7FFFFFFFLL)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "%d sequences of %d heads of %d columns: above 2^31 - 1 blocks", g.q.n_seq,
                        d.heads, d.dv);
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;

    g.qp = q, g.kp = k, g.vp = v, g.dt = dt, g.b = b, g.a = a, g.dt_bias = dt_bias, g.state_in = state_in;
    g.y = y, g.state_out = state_out;
    g.ld_q = d.ld_q, g.ld_k = d.ld_k, g.ld_v = d.ld_v, g.ld_dt = d.ld_dt, g.ld_b = d.ld_b, g.ld_y = d.ld_y;
    g.heads = d.heads, g.per_key = d.heads / d.key_heads, g.dk = d.dk, g.dv = d.dv;
    g.softplus = d.softplus, g.sigmoid = d.sigmoid, g.normalize = d.normalize, g.scale = d.scale;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t ce = d.dtype == FCM_F32   ? seq::run_delta<float>(g, cs)
                           : d.dtype == FCM_F16 ? seq::run_delta<__half>(g, cs)
                                                : seq::run_delta<__nv_bfloat16>(g, cs);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
