// seq_scan.cu -- the selective scan: argument checks, the choice of kernel, and the kernel for
// single tokens.  The kernel for prompts is in seq_scan.cuh.
#include <math.h>

#include "seq_scan.cuh"

namespace fcm {
namespace seq {

struct TokenArgs {
    Seqs q;
    const void *x, *dt, *bm, *cm, *z;
    const float *a, *skip, *dt_bias, *state_in;
    void *y;
    float *state_out;
    int ld_x, ld_dt, ld_b, ld_c, ld_z, ld_y;
    int c, n, cpg, softplus;
    int blocks;   // of channels
    int turns;    // blocks per block of channels: each takes every turns-th pair of sequences
};

// p's row of `ld` elements: one 32 x 32 bit product.
template <typename T> __device__ __forceinline__ const T *row_of(const void *p, int row, int ld) {
    return static_cast<const T *>(p) + (long long)row * ld;
}

// Sequences of at most one row: what counts is the states' way through the chip and back.  A thread
// has four states of one channel (LPC lanes have all n), of two sequences at a time; its block goes
// from pair to pair, and a pair's states, B, C, x, dt and z are loaded while the pair before is
// computed (the slots that say where, one pair earlier).  Loads are unconditional, so that they are
// all under way at once: what does not exist is read from a place that does, and not used.  The
// steps and gates are made once per channel, by the block's threads together.  VEC: the states, a,
// bm and cm are read, and the states written, four at a time.
//
// Bound by memory: 192 sequences x 5120 channels x 16 states, 134 MB read and written in 33.5 us, 4.0
// TB/s, 0.60 of a plain copy's rate; a kernel that only multiplies 63 MB of states takes 20 us here, so
// that what remains is the issue (64 % of the cycles: the products' addresses and the sums over lanes).
// A single sequence of 1536 channels takes 2.2 us, a launch.
template <typename T, bool VEC, int LPC>
__global__ void __launch_bounds__(128, 6) scan_token_kernel(const TokenArgs a) {
    constexpr int U = 2, CHANS = 128 / LPC;
    __shared__ float4 prep[2][U * CHANS];   // step, step * x, skip * x, gate of [sequence][channel]
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int n0 = 4 * (threadIdx.x % LPC), ch = threadIdx.x / LPC;
    const unsigned channels = a.c, d0 = blockIdx.x % a.blocks * CHANS;   // past 2^31 with a block's added
    const int d = (int)min(d0 + ch, channels - 1);
    const bool live = d0 + ch < channels, some = a.q.tokens > 0, mine = VEC ? n0 < a.n : true;
    const int last = (int)a.q.tokens - 1;
    // the sequence and channel whose step this thread makes
    const int pu = min((int)threadIdx.x / CHANS, U - 1), pd = (int)min(d0 + threadIdx.x % CHANS, channels - 1);
    const bool makes = (int)threadIdx.x < U * CHANS;
    const float bias = a.dt_bias ? a.dt_bias[pd] : 0.0f, skip = a.skip ? a.skip[pd] : 0.0f;

    // four elements from n0 on (p: of the state that is read first), or the last one in the place
    // of those past n
    const int nl = VEC ? min(n0, a.n - 4) : min(n0, a.n - 1);
    auto four = [&](auto &to, const auto *p) {
        typedef typename std::remove_const<typename std::remove_pointer<decltype(p)>::type>::type E;
        if (VEC) {
            to = *reinterpret_cast<const Vec<E, 4> *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) to.e[i] = p[min(i, a.n - 1 - nl)];
        }
    };
    const int cn = a.c * a.n, gn = d / a.cpg * a.n + nl;
    const float *state_in = a.state_in + (size_t)d * a.n + nl;
    float *state_out = a.state_out + (size_t)d * a.n + n0;
    const T *bm = static_cast<const T *>(a.bm) + gn, *cm = static_cast<const T *>(a.cm) + gn;
    T *y = static_cast<T *>(a.y) + d;
    Vec<float, 4> av;
    four(av, a.a + (size_t)d * a.n + nl);
#pragma unroll
    for (int i = 0; i < 4; i++) av.e[i] *= kLog2e;

    struct Where {
        int t[U], len[U], row[U];   // len -1: there is no such sequence
    };
    auto look = [&](int q0) {
        Where w;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int q = min(q0 + u, a.q.n_seq - 1);
            long long t;
            seq_rows(a.q, q, t, w.len[u]);
            w.t[u] = min((int)t, last);
            if (q0 + u >= a.q.n_seq) w.len[u] = -1;
            w.row[u] = a.state_in || a.state_out ? state_row(a.q, q) : -1;
        }
        return w;
    };
    struct Loads {
        Vec<float, 4> h[U];
        Vec<T, 4> b[U], c[U];
        T x, dt, z;
    };
    auto load = [&](const Where &w, Loads &v) {
        if (a.state_in) {
#pragma unroll
            for (int u = 0; u < U; u++) four(v.h[u], row_of<float>(state_in, max(w.row[u], 0), cn));
        }
        if (some) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                four(v.b[u], row_of<T>(bm, w.t[u], a.ld_b));
                four(v.c[u], row_of<T>(cm, w.t[u], a.ld_c));
            }
            const int at = pu ? w.t[1] : w.t[0];
            v.x = row_of<T>(a.x, at, a.ld_x)[pd];
            v.dt = row_of<T>(a.dt, at, a.ld_dt)[pd];
            if (a.z) v.z = row_of<T>(a.z, at, a.ld_z)[pd];
        }
    };
    const int stride = U * a.turns;
    int q0 = (int)(blockIdx.x / a.blocks) * U;
    Where where = look(q0), then = look(q0 + stride);
    Loads now, next;
    load(where, now);
    for (int turn = 0; q0 < a.q.n_seq; q0 += stride, turn ^= 1) {
        if (q0 + stride < a.q.n_seq) load(then, next);
        const Where after = look(q0 + 2 * stride);
        if (makes && some) {
            const float x = Storage<T>::to_f(now.x);
            float step = Storage<T>::to_f(now.dt) + bias, unused = 0.0f;
            if (a.softplus) softplus2(step, unused);
            prep[turn][threadIdx.x] = make_float4(step, step * x, a.skip ? skip * x : 0.0f,
                                                  a.z ? silu(Storage<T>::to_f(now.z)) : 1.0f);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; u++) {
            Vec<float, 4> h = now.h[u];
            if (!a.state_in || where.row[u] < 0)
#pragma unroll
                for (int i = 0; i < 4; i++) h.e[i] = 0.0f;
            if (where.len[u] > 0) {
                const float4 p = prep[turn][u * CHANS + ch];
                float bv[4], cv[4], o = 0.0f;
                now.b[u].get(bv);
                now.c[u].get(cv);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    h.e[i] = fmaf(ex2(p.x * av.e[i]), h.e[i], p.y * bv[i]);
                    if (VEC || n0 + i < a.n) o = fmaf(cv[i], h.e[i], o);
                }
                o = mine ? o : 0.0f;
#pragma unroll
                for (int m = 1; m < LPC; m *= 2) o += __shfl_xor_sync(0xFFFFFFFFu, o, m);
                if (n0 == 0 && live) y[(long long)where.t[u] * a.ld_y] = Storage<T>::from_f((o + p.z) * p.w);
            }
            if (where.len[u] >= 0 && where.row[u] >= 0 && a.state_out && live) {
                float *to = state_out + (long long)where.row[u] * cn;
                if (VEC) {
                    if (mine) *reinterpret_cast<Vec<float, 4> *>(to) = h;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (n0 + i < a.n) to[i] = h.e[i];
                }
            }
        }
        now = next, where = then, then = after;
    }
}

template <typename T, int LPC>
static cudaError_t launch_tokens(TokenArgs t, int sms, bool vec, cudaStream_t st) {
    constexpr int CHANS = 128 / LPC;
    t.blocks = (t.c - 1) / CHANS + 1;
    // A few blocks for each place an SM has, or as many as there are pairs.  Measured, us with 3, 6, 12, 24,
    // 48 blocks an SM: 192 x 5120 67.6, 36.5, 33.7, 35.6, 38.4; 64 x 4096 12.7, 9.8, 9.7, 11.5, 11.9; 160 x 1536 11.3, 8.5,
    // 9.2, 11.1, 11.2.
    const long long pairs = (t.q.n_seq + 1) / 2, room = (long long)sms * 12 / t.blocks;
    t.turns = (int)(pairs < room ? pairs : room > 1 ? room : 1);
    const long long grid = (long long)t.blocks * t.turns;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
    return launch(vec ? scan_token_kernel<T, true, LPC> : scan_token_kernel<T, false, LPC>, dim3((unsigned)grid),
                  128, 0, st, t);
}

template <typename T>
static cudaError_t run_tokens(const ScanArgs &a, int sms, cudaStream_t st) {
    const TokenArgs t = {a.q, a.x, a.dt, a.bm, a.cm, a.z, a.a, a.skip, a.dt_bias, a.state_in, a.y, a.state_out,
                         (int)a.ld_x, (int)a.ld_dt, (int)a.ld_b, (int)a.ld_c, (int)a.ld_z, (int)a.ld_y,
                         a.c, a.n, a.cpg, a.softplus, 0, 0};
    const size_t four = 4 * sizeof(T);
    const bool vec = a.n % 4 == 0 && aligned16(a.a) && aligned16(a.state_in) && aligned16(a.state_out) &&
                     reinterpret_cast<uintptr_t>(a.bm) % four == 0 && reinterpret_cast<uintptr_t>(a.cm) % four == 0 &&
                     a.ld_b % 4 == 0 && a.ld_c % 4 == 0;
    if (a.n <= 8) return launch_tokens<T, 2>(t, sms, vec, st);
    if (a.n <= 16) return launch_tokens<T, 4>(t, sms, vec, st);
    if (a.n <= 32) return launch_tokens<T, 8>(t, sms, vec, st);
    if (a.n <= 64) return launch_tokens<T, 16>(t, sms, vec, st);
    return launch_tokens<T, 32>(t, sms, vec, st);
}

// Which shape scans, and over how many parts a sequence is split.  More states per thread cost
// less per state but leave fewer blocks and more serial work; parts run side by side, but all but
// the last go over their rows twice.  Measured on one GB300, nanoseconds per row of a block that
// has its SM to itself (t1); two blocks of an SM take 1.74 times that, or twice it where their
// shared memory only lets one in at a time; splitting costs 1.69 times the rows, and 4 us; clusters of
// eight are put on fewer SMs, so that 16 of them (128 blocks) are pairs already, 12 are not.
// Against the other shapes and parts, bf16, 16 states, us (4x4, 8x2, 16x1 states x lanes):
//   1 x 8192 rows x 4096 channels:  whole 245, 400, 797; best split 339 (2), 329 (8), 340 (8)
//   1 x 8192 x 1024:                whole 245, 400, 797; best split  98 (8), 151 (8), 175 (8)
//   4 x 2048 x 4096:                whole 215, 176, 203; split from 269
//   32 x 256 x 4096:                whole 199, 160, 157; split from 271
struct ScanChoice {
    int spt, lpc, parts;
};
template <typename T> static ScanChoice choose_scan(const ScanArgs &a, int sms) {
    static constexpr struct {
        int spt, lpc, most, exact;   // states it takes; exact: no fewer
        double t1;
    } shapes[] = {{4, 1, 4, 0, 80.0},  {4, 2, 8, 0, 43.1},   {4, 4, 16, 0, 30.3}, {8, 2, 16, 1, 48.9},
                  {16, 1, 16, 1, 97.3}, {4, 8, 32, 0, 33.5}, {8, 4, 32, 1, 44.0}, {8, 8, 64, 0, 49.3},
                  {8, 16, 128, 0, 60.0}};
    ScanChoice best = {8, 16, 1};
    double least = 1e300;
    int most = 0;   // the narrowest width that holds the states
    for (const auto &s : shapes)
        if (s.most >= a.n && (most == 0 || s.most < most)) most = s.most;
    const double rows = (double)a.q.max_len, filled = a.q.seq_start && a.q.n_seq
        ? (double)a.q.tokens / ((double)a.q.n_seq * rows) : 1.0;
    for (const auto &s : shapes) {
        if (s.most != most || (s.exact && a.n != s.most)) continue;
        const int ch = 4 * (32 / s.lpc);
        const double pair = 2 * scan_smem<T>(s.spt, s.lpc) <= 227 * 1024 ? 1.74 : 2.0;
        for (int parts = 1; parts <= 8; parts *= 2) {
            const double blocks = (double)a.q.n_seq * a.groups * ((a.cpg - 1) / ch + 1) * parts;
            const double load = ceil(blocks * (filled < 1.0 ? filled : 1.0) / (2.0 * sms));
            const bool alone = parts == 8 ? 4 * blocks <= 3.0 * sms : blocks <= sms;
            const double step = alone ? s.t1 : s.t1 * pair * (load > 1.0 ? load : 1.0);
            const double ns = parts == 1 ? step * rows : 1.69 * step * rows / parts + 4000.0;
            if (ns < least) least = ns, best = {s.spt, s.lpc, parts};
        }
    }
    return best;
}

template <typename T>
static cudaError_t run_scan(const ScanArgs &a, int sms, cudaStream_t st) {
    if (a.q.max_len <= 1) return run_tokens<T>(a, sms, st);
    const ScanChoice c = choose_scan<T>(a, sms);
    return launch_scan<T>(a, c.spt, c.lpc, c.parts, st);
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_selective_scan(const fcm_scan_desc *desc, const void *x, const void *dt,
                                         const float *a, const void *bm, const void *cm,
                                         const float *skip, const void *z, const float *dt_bias,
                                         const float *state_in, void *y, float *state_out,
                                         void *stream) {
    FcmNvtxRange nvtx("fcm_selective_scan");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_scan_desc d = *desc;
    if (d.c < 1 || d.n_state < 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "c %d, n_state %d", d.c, d.n_state);
    if (d.n_state > seq::kMaxState)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "n_state %d above %d", d.n_state, seq::kMaxState);
    if ((long long)d.c * d.n_state > 0x7FFFFFFFLL)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "c * n_state above 2^31 - 1");
    if (d.groups < 1 || d.c % d.groups)
        return fcm_fail(FCM_ERR_INVALID_ARG, "%d groups do not divide %d channels", d.groups, d.c);
    if (d.dtype < FCM_F32 || d.dtype > FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d.dtype);
    if (d.softplus != 0 && d.softplus != 1)
        return fcm_fail(FCM_ERR_INVALID_ARG, "softplus %d: 0 or 1", d.softplus);
    seq::ScanArgs k = {};
    const long long bc = (long long)d.groups * d.n_state;
    fcm_status st;
    if ((st = seq::check_seqs(d.seqs, state_in || state_out, &k.q)) != FCM_OK ||
        (st = seq::check_ld(&d.ld_x, d.c, "ld_x")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_dt, d.c, "ld_dt")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_b, bc, "ld_b")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_c, bc, "ld_c")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_z, d.c, "ld_z")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_y, d.c, "ld_y")) != FCM_OK)
        return st;
    if (k.q.n_seq == 0) return FCM_OK;
    const size_t e = (size_t)fcm_dtype_bytes(d.dtype);
    const long long rows = k.q.tokens;   // without rows the activations may be NULL
    if ((rows && ((st = seq::check_dev_ptr(x, e, "x")) != FCM_OK ||
                  (st = seq::check_dev_ptr(dt, e, "dt")) != FCM_OK ||
                  (st = seq::check_dev_ptr(bm, e, "bm")) != FCM_OK ||
                  (st = seq::check_dev_ptr(cm, e, "cm")) != FCM_OK ||
                  (st = seq::check_dev_ptr(y, e, "y")) != FCM_OK)) ||
        (z && (st = seq::check_dev_ptr(z, e, "z")) != FCM_OK) ||
        (st = seq::check_dev_ptr(a, 4, "a")) != FCM_OK ||
        (skip && (st = seq::check_dev_ptr(skip, 4, "skip")) != FCM_OK) ||
        (dt_bias && (st = seq::check_dev_ptr(dt_bias, 4, "dt_bias")) != FCM_OK) ||
        (state_in && (st = seq::check_dev_ptr(state_in, 4, "state_in")) != FCM_OK) ||
        (state_out && (st = seq::check_dev_ptr(state_out, 4, "state_out")) != FCM_OK))
        return st;
    const struct {
        const void *p;
        long long ld, cols;
        const char *name;
    } ins[] = {{x, d.ld_x, d.c, "x"}, {dt, d.ld_dt, d.c, "dt"}, {bm, d.ld_b, bc, "bm"},
               {cm, d.ld_c, bc, "cm"}, {z, d.ld_z, d.c, "z"}};
    for (const auto &in : ins)
        if (seq::rows_overlap(in.p, in.ld, in.cols, y, d.ld_y, d.c, rows, e))
            return fcm_fail(FCM_ERR_INVALID_ARG, "%s and y overlap", in.name);
    const long long state_row = (long long)d.c * d.n_state;
    if (state_in != state_out &&
        seq::rows_overlap(state_in, state_row, state_row, state_out, state_row, state_row, k.q.slots, 4))
        return fcm_fail(FCM_ERR_INVALID_ARG, "state_in and state_out overlap without being the same");
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;

    k.x = x, k.dt = dt, k.bm = bm, k.cm = cm, k.z = z, k.a = a, k.skip = skip, k.dt_bias = dt_bias;
    k.state_in = state_in, k.y = y, k.state_out = state_out;
    k.ld_x = d.ld_x, k.ld_dt = d.ld_dt, k.ld_b = d.ld_b, k.ld_c = d.ld_c, k.ld_z = d.ld_z, k.ld_y = d.ld_y;
    k.c = d.c, k.n = d.n_state, k.groups = d.groups, k.softplus = d.softplus;
    k.cpg = d.c / d.groups;
    const size_t e16 = 16 / e;
    const long long starts = d.groups == 1 ? 0 : k.cpg | d.n_state;   // a group's first column
    k.vec16 = seq::aligned16(x) && seq::aligned16(dt) && seq::aligned16(z) &&
              ((d.ld_x | d.ld_dt | (z ? d.ld_z : 0) | (d.groups == 1 ? 0 : k.cpg)) % e16) == 0;
    k.vec16n = seq::aligned16(bm) && seq::aligned16(cm) &&
               ((d.ld_b | d.ld_c | (d.groups == 1 ? 0 : d.n_state)) % e16) == 0;
    k.vec2 = reinterpret_cast<uintptr_t>(y) % (2 * e) == 0 && (d.ld_y | starts) % 2 == 0;
    const cudaError_t ce = d.dtype == FCM_F32   ? seq::run_scan<float>(k, sms, static_cast<cudaStream_t>(stream))
                           : d.dtype == FCM_F16 ? seq::run_scan<__half>(k, sms, static_cast<cudaStream_t>(stream))
                                                : seq::run_scan<__nv_bfloat16>(k, sms, static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
