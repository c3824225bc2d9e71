// seq_scan.cu -- the selective scan: argument checks, the choice of kernel, and the kernel for
// single tokens.  The kernel for prompts is in seq_scan.cuh.
#include "seq_scan.cuh"

namespace fcm {
namespace seq {

struct TokenArgs {
    ScanArgs s;
    int lpc;      // lanes per channel, a power of two, 4 * lpc >= n
    int chunks;   // times a thread takes U sequences
};

// Sequences of at most one row.  A thread has four states of one channel and takes U sequences at
// a time: it reads all that they need before it writes anything.  VEC: the states, a, bm and cm
// are read four at a time.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(128) scan_token_kernel(const TokenArgs ta) {
    const ScanArgs &a = ta.s;
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const int lpc = ta.lpc, part = threadIdx.x % lpc, n0 = 4 * part;
    const int d = blockIdx.x * (128 / lpc) + threadIdx.x / lpc;
    const bool live = d < a.c;
    const int dd = live ? d : 0, g = dd / a.cpg;
    bool in[4];
    float av[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        in[i] = live && (VEC ? n0 < a.n : n0 + i < a.n);
        av[i] = in[i] ? a.a[(size_t)dd * a.n + n0 + i] * kLog2e : 0.0f;
    }
    const float bias = a.dt_bias ? a.dt_bias[dd] : 0.0f, skip = a.skip ? a.skip[dd] : 0.0f;
    for (int chunk = 0; chunk < ta.chunks; chunk++) {
        const int q0 = (blockIdx.y * ta.chunks + chunk) * U;
        if (q0 >= a.q.n_seq) break;
        float h[U][4], b[U][4], c[U][4], x[U], dt[U], z[U];
        long long t[U];
        int len[U], row[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            len[u] = 0, row[u] = -1, t[u] = 0;
            x[u] = dt[u] = z[u] = 0.0f;
            if (q0 + u < a.q.n_seq) {
                seq_rows(a.q, q0 + u, t[u], len[u]);
                if (a.state_in || a.state_out) row[u] = state_row(a.q, q0 + u);
            }
            const float *hp = a.state_in + ((size_t)(row[u] < 0 ? 0 : row[u]) * a.c + dd) * a.n + n0;
            const T *bp = static_cast<const T *>(a.bm) + t[u] * a.ld_b + (long long)g * a.n + n0;
            const T *cp = static_cast<const T *>(a.cm) + t[u] * a.ld_c + (long long)g * a.n + n0;
            const bool some = len[u] > 0 && live;
#pragma unroll
            for (int i = 0; i < 4; i++) h[u][i] = b[u][i] = c[u][i] = 0.0f;
            if (VEC) {
                if (in[0] && row[u] >= 0 && a.state_in) {
                    const float4 v = *reinterpret_cast<const float4 *>(hp);
                    h[u][0] = v.x, h[u][1] = v.y, h[u][2] = v.z, h[u][3] = v.w;
                }
                if (in[0] && some) {
                    reinterpret_cast<const Vec<T, 4> *>(bp)->get(b[u]);
                    reinterpret_cast<const Vec<T, 4> *>(cp)->get(c[u]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (in[i] && row[u] >= 0 && a.state_in) h[u][i] = hp[i];
                    if (in[i] && some) {
                        b[u][i] = Storage<T>::to_f(bp[i]);
                        c[u][i] = Storage<T>::to_f(cp[i]);
                    }
                }
            }
            if (some) {
                x[u] = Storage<T>::to_f(static_cast<const T *>(a.x)[t[u] * a.ld_x + d]);
                dt[u] = Storage<T>::to_f(static_cast<const T *>(a.dt)[t[u] * a.ld_dt + d]);
                if (a.z) z[u] = Storage<T>::to_f(static_cast<const T *>(a.z)[t[u] * a.ld_z + d]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            float step = dt[u] + bias;
            if (a.softplus) {
                float unused = 0.0f;
                softplus2(step, unused);
            }
            const float du = step * x[u];
            float o = 0.0f;
            if (len[u] > 0) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (!in[i]) continue;   // a padding state's 0 * infinity stays out of the sum
                    h[u][i] = fmaf(ex2(step * av[i]), h[u][i], du * b[u][i]);
                    o = fmaf(c[u][i], h[u][i], o);
                }
            }
            for (int m = 1; m < lpc; m *= 2) o += __shfl_xor_sync(0xFFFFFFFFu, o, m);
            if (part == 0 && live && len[u] > 0) {
                if (a.skip) o = fmaf(skip, x[u], o);
                if (a.z) o *= silu(z[u]);
                static_cast<T *>(a.y)[t[u] * a.ld_y + d] = Storage<T>::from_f(o);
            }
            if (row[u] >= 0 && a.state_out) {
                float *hp = a.state_out + ((size_t)row[u] * a.c + dd) * a.n + n0;
                if (VEC) {
                    if (in[0]) *reinterpret_cast<float4 *>(hp) = make_float4(h[u][0], h[u][1], h[u][2], h[u][3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (in[i]) hp[i] = h[u][i];
                }
            }
        }
    }
}

template <typename T>
static cudaError_t run_tokens(const ScanArgs &a, int sms, cudaStream_t st) {
    TokenArgs t = {a, 1, 1};
    while (4 * t.lpc < a.n) t.lpc *= 2;
    const size_t four = 4 * sizeof(T);
    const bool vec = a.n % 4 == 0 && aligned16(a.state_in) && aligned16(a.state_out) &&
                     reinterpret_cast<uintptr_t>(a.bm) % four == 0 && reinterpret_cast<uintptr_t>(a.cm) % four == 0 &&
                     a.ld_b % 4 == 0 && a.ld_c % 4 == 0;
    const unsigned gx = (unsigned)((a.c + 128 / t.lpc - 1) / (128 / t.lpc));
    const bool many = (long long)gx * a.q.n_seq >= (long long)sms * 64;
    const int u = many ? 4 : 1;
    t.chunks = many ? 2 : 1;
    const long long gy = (a.q.n_seq + (long long)u * t.chunks - 1) / (u * t.chunks);
    if (gy > 65535) {
        t.chunks = (int)((a.q.n_seq + 65535LL * u - 1) / (65535LL * u));
    }
    const unsigned gyy = (unsigned)((a.q.n_seq + (long long)u * t.chunks - 1) / ((long long)u * t.chunks));
    void (*kernel)(TokenArgs) = vec ? (many ? scan_token_kernel<T, true, 4> : scan_token_kernel<T, true, 1>)
                                    : (many ? scan_token_kernel<T, false, 4> : scan_token_kernel<T, false, 1>);
    return launch(kernel, dim3(gx, gyy), 128, 0, st, t);
}

// Which shape scans, and over how many parts a sequence is split.  More states per thread cost
// less per state but leave fewer blocks and more serial work; parts run side by side, but all but
// the last go over their rows twice.  Measured on one GB300, nanoseconds per row of a block that
// has its SM to itself (t1); two blocks of an SM take 1.68 times that, or twice it where their
// shared memory only lets one in at a time; splitting costs 1.69 times the rows, and 4 us.
// Against the other shapes and parts, bf16, 16 states, us (4x4, 8x2, 16x1 states x lanes):
//   1 x 8192 rows x 4096 channels:  whole 282, 464, 857; best split 364 (2), 328 (4), 322 (8)
//   1 x 8192 x 1024:                whole 282, 464, 856; best split  99 (8), 156 (8), 184 (8)
//   4 x 2048 x 4096:                whole 233, 187, 216; split from 279
//   32 x 256 x 4096:                whole 208, 168, 162; split from 270
struct ScanChoice {
    int spt, lpc, parts;
};
template <typename T> static ScanChoice choose_scan(const ScanArgs &a, int sms) {
    static constexpr struct {
        int spt, lpc, most, exact;   // states it takes; exact: no fewer
        double t1;
    } shapes[] = {{4, 1, 4, 0, 80.0},  {4, 2, 8, 0, 50.0},   {4, 4, 16, 0, 34.4}, {8, 2, 16, 1, 56.6},
                  {16, 1, 16, 1, 104.5}, {4, 8, 32, 0, 36.8}, {8, 4, 32, 1, 47.7}, {8, 8, 64, 0, 50.0},
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
        const double pair = 2 * scan_smem<T>(s.spt, s.lpc) <= 227 * 1024 ? 1.68 : 2.0;
        for (int parts = 1; parts <= 8; parts *= 2) {
            const double blocks = (double)a.q.n_seq * a.groups * ((a.cpg + ch - 1) / ch) * parts;
            const double load = blocks * (filled < 1.0 ? filled : 1.0) / (2.0 * sms);
            const double step = blocks <= sms ? s.t1 : s.t1 * pair * (load > 1.0 ? load : 1.0);
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
    k.vec16 = seq::aligned16(x) && seq::aligned16(dt) && seq::aligned16(bm) && seq::aligned16(cm) &&
              seq::aligned16(z) && ((d.ld_x | d.ld_dt | d.ld_b | d.ld_c | (z ? d.ld_z : 0) | starts) % e16) == 0;
    k.vec2 = reinterpret_cast<uintptr_t>(y) % (2 * e) == 0 && (d.ld_y | starts) % 2 == 0;
    const cudaError_t ce = d.dtype == FCM_F32   ? seq::run_scan<float>(k, sms, static_cast<cudaStream_t>(stream))
                           : d.dtype == FCM_F16 ? seq::run_scan<__half>(k, sms, static_cast<cudaStream_t>(stream))
                                                : seq::run_scan<__nv_bfloat16>(k, sms, static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
