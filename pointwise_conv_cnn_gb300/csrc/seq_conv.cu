// seq_conv.cu -- causal depthwise convolution over sequences with its cached rows.
//
// y[i,d] = act(s[d] * sum_j w[d,j] * xx[i+j,d] + b[d]), xx = the k-1 cached rows, then x.
#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

struct ConvArgs {
    Seqs q;
    const void *x, *w;
    const float *s, *b;
    const void *state_in;
    void *y, *state_out;
    long long ld_x, ld_y;
    int c, k, act;
    int rows;      // output rows per thread
    int tiles;     // tiles of `rows` rows that cover max_len
    long long threads;
};

constexpr int kMaxTaps = 8;

// VEC elements of x or of one tap's weights as the products take them: two 16-bit ones in a register
// (fma.rn.f32.{f16,bf16} widens both factors), or single ones widened.
template <typename T, int VEC> struct Lane {
    static constexpr bool PACKED = sizeof(T) == 2 && VEC > 1;
    static constexpr int N = PACKED ? VEC / 2 : VEC;
    typedef typename std::conditional<PACKED, uint32_t, float>::type R;
    R r[N];
    struct alignas(VEC * sizeof(T)) Bits {
        uint32_t u[VEC * sizeof(T) >= 4 ? VEC * sizeof(T) / 4 : 1];
    };
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC == 1) {
            r[0] = Storage<T>::to_f(*p);
        } else {
            const Bits v = *reinterpret_cast<const Bits *>(p);
#pragma unroll
            for (int i = 0; i < N; i++) r[i] = from_bits(v.u[i]);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (VEC == 1) {
            *p = Storage<T>::from_f(r[0]);
        } else {
            Bits v;
#pragma unroll
            for (int i = 0; i < N; i++) v.u[i] = to_bits(r[i]);
            *reinterpret_cast<Bits *>(p) = v;
        }
    }
    static __device__ __forceinline__ R from_bits(uint32_t u) {
        if constexpr (PACKED) return u;
        else return __uint_as_float(u);
    }
    static __device__ __forceinline__ uint32_t to_bits(R v) {
        if constexpr (PACKED) return v;
        else return __float_as_uint(v);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; i++) r[i] = 0;
    }
    // element v of this lane's channels from a value in memory
    __device__ __forceinline__ void set(int v, T value) {
        if constexpr (PACKED) {
            const uint32_t bits = *reinterpret_cast<const unsigned short *>(&value);
            r[v / 2] = v % 2 ? (r[v / 2] & 0xFFFFu) | bits << 16 : bits;
        } else {
            r[v] = Storage<T>::to_f(value);
        }
    }
    __device__ __forceinline__ void multiply_add(float (&acc)[VEC], const Lane &w) const {
        if constexpr (PACKED) {
#pragma unroll
            for (int i = 0; i < N; i++) tc::Fma16<T>::fma2(acc[2 * i], acc[2 * i + 1], r[i], w.r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) acc[i] = fmaf(w.r[i], r[i], acc[i]);
        }
    }
};

// One thread: VEC neighbouring channels (16 bytes, or one), a.rows consecutive rows of one
// sequence.  The K - 1 rows before them are read again from the neighbour's tile or are the cached
// ones; from there each row is read once and kept in registers, as stored, for its K uses.  The
// thread of a sequence's first rows also replaces the cached rows, which it has read by then, so
// that state_out may be state_in.
//
// Bound by memory where rows are 16-byte aligned: 16384 x 4096 bf16, 4 taps and silu, 268 MB in 50.3 us,
// 5.3 TB/s, 0.80 of a plain copy's rate (what is left: the first rows' and the weights' loads, which a
// tile waits for before its first product).  One channel a thread is bound by what it issues, 28
// instructions an element: 16384 x 4095 67.9 us.  A single token is a launch: 1536 channels 2.2 us.
template <typename T, int VEC, int K>
__global__ void __launch_bounds__(128) causal_conv_kernel(const ConvArgs a) {
    typedef Lane<T, VEC> L;
    constexpr int H = K - 1, U = 8;   // rows before, rows loaded at once
    tc::pdl_wait();
    tc::pdl_launch_dependents();
    const long long id = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= a.threads) return;
    const int cg = a.c / VEC, d = (int)(id % cg) * VEC;
    const long long rest = id / cg;
    const int tile = (int)(rest % a.tiles), q = (int)(rest / a.tiles);
    long long start;
    int len;
    seq_rows(a.q, q, start, len);
    const unsigned i0 = (unsigned)tile * a.rows, i1 = min((unsigned)len, i0 + a.rows);   // may pass 2^31 with rows added
    if (tile > 0 && i0 >= i1) return;
    const T *x = static_cast<const T *>(a.x) + d + start * a.ld_x;
    T *y = static_cast<T *>(a.y) + d + start * a.ld_y;

    L win[H + U];   // rows i - H .. i + U - 1
    int row = -1;
    size_t at = 0;
    if (K > 1) {
        if (tile == 0) {
            if (a.state_in || a.state_out) row = state_row(a.q, q);
            at = (size_t)(row < 0 ? 0 : row) * H * a.c + d;
#pragma unroll
            for (int j = 0; j < H; j++) {
                win[j].zero();
                if (row >= 0 && a.state_in) win[j].load(static_cast<const T *>(a.state_in) + at + (size_t)j * a.c);
            }
        } else {
#pragma unroll
            for (int j = 0; j < H; j++) win[j].load(x + (long long)(i0 - H + j) * a.ld_x);
        }
    }
    L w[K];
    float s[VEC], b[VEC];
    {
        constexpr int PIECE = VEC * K * sizeof(T) % 16 == 0 && VEC > 2 ? 16 / (int)sizeof(T) : 1;   // w's own order
#pragma unroll
        for (int j = 0; j < VEC * K; j += PIECE) {
            const Vec<T, PIECE> p = *reinterpret_cast<const Vec<T, PIECE> *>(static_cast<const T *>(a.w) + (size_t)d * K + j);
#pragma unroll
            for (int v = 0; v < PIECE; v++) w[(j + v) % K].set((j + v) / K, p.e[v]);
        }
#pragma unroll
        for (int v = 0; v < VEC; v++) s[v] = 1.0f, b[v] = 0.0f;
        constexpr int F = VEC % 4 == 0 ? 4 : VEC;
#pragma unroll
        for (int v = 0; v < VEC; v += F) {
            if (a.s) {
                const Vec<float, F> p = *reinterpret_cast<const Vec<float, F> *>(a.s + d + v);
#pragma unroll
                for (int e = 0; e < F; e++) s[v + e] = p.e[e];
            }
            if (a.b) {
                const Vec<float, F> p = *reinterpret_cast<const Vec<float, F> *>(a.b + d + v);
#pragma unroll
                for (int e = 0; e < F; e++) b[v + e] = p.e[e];
            }
        }
    }
    // The state after: the last H places, of which those before 0 are cached rows.  All are read
    // before any is written.
    if (K > 1 && row >= 0 && a.state_out) {
        L last[K > 1 ? H : 1];
#pragma unroll
        for (int j = 0; j < H; j++) {
            const int i = len - H + j;
            last[j].zero();
            if (i >= 0) last[j].load(x + (long long)i * a.ld_x);
            else if (a.state_in) last[j].load(static_cast<const T *>(a.state_in) + at + (size_t)(i + H) * a.c);
        }
#pragma unroll
        for (int j = 0; j < H; j++) last[j].store(static_cast<T *>(a.state_out) + at + (size_t)j * a.c);
    }
    // the rows' addresses by addition: a product each would be half of a single channel's instructions
    const T *from = x + (long long)i0 * a.ld_x;
    T *to = y + (long long)i0 * a.ld_y;
    auto compute = [&](int n) {   // the n rows that were loaded
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (u >= n) break;
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; v++) o[v] = 0.0f;
#pragma unroll
            for (int j = 0; j < K; j++) win[u + j].multiply_add(o, w[j]);
#pragma unroll
            for (int v = 0; v < VEC; v++) o[v] = fmaf(s[v], o[v], b[v]);
            if (a.act == FCM_ACT_SILU) {
#pragma unroll
                for (int v = 0; v < VEC; v++) o[v] = silu(o[v]);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; v++) o[v] = clamp_act(o[v], a.act);
            }
            Vec<T, VEC> out;
            out.put(o);
            *reinterpret_cast<Vec<T, VEC> *>(to) = out;
            to += a.ld_y;
        }
#pragma unroll
        for (int j = 0; j < H; j++) win[j] = win[U + j];
    };
    unsigned i = i0;
    for (; i + U <= i1; i += U) {
#pragma unroll
        for (int u = 0; u < U; u++, from += a.ld_x) win[H + u].load(from);
        compute(U);
    }
    if (i + 1 < i1) {   // the last one again in the place of rows that there are not: no load waits
#pragma unroll
        for (int u = 0; u < U; u++) {
            win[H + u].load(from);
            if (i + u + 1 < i1) from += a.ld_x;
        }
        compute((int)(i1 - i));
    } else if (i < i1) {
        win[H].load(from);
        compute(1);
    }
}

template <typename T, int VEC>
static void (*pick_conv(int k))(ConvArgs) {
    switch (k) {
    case 1: return causal_conv_kernel<T, VEC, 1>;
    case 2: return causal_conv_kernel<T, VEC, 2>;
    case 3: return causal_conv_kernel<T, VEC, 3>;
    case 4: return causal_conv_kernel<T, VEC, 4>;
    case 5: return causal_conv_kernel<T, VEC, 5>;
    case 6: return causal_conv_kernel<T, VEC, 6>;
    case 7: return causal_conv_kernel<T, VEC, 7>;
    default: return causal_conv_kernel<T, VEC, 8>;
    }
}

template <typename T>
static cudaError_t run_conv(ConvArgs a, int sms, cudaStream_t st) {
    constexpr int VEC = 16 / (int)sizeof(T);
    // 16 bytes a thread where every row allows it, else two channels, else one.  Measured, bf16, 4 taps,
    // us with 8, 2, 1 channels: 16384 x 4096 50.7, 49.3, 68.0; 1024 x 2048 4.0, 4.9, 5.0; 256 single tokens x
    // 5120 6.8, 8.1, 14.3.
    auto rows_allow = [&](int n) {
        const size_t bytes = n * sizeof(T);
        auto fits = [](const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; };
        return ((a.c | a.ld_x | a.ld_y) % n) == 0 && fits(a.x, bytes) && fits(a.y, bytes) && fits(a.state_in, bytes) &&
               fits(a.state_out, bytes) && fits(a.w, n > 2 ? 16 : sizeof(T)) && fits(a.s, n > 2 ? 16 : 8) &&
               fits(a.b, n > 2 ? 16 : 8);
    };
    const int vec = rows_allow(VEC) ? VEC : rows_allow(2) ? 2 : 1;
    const long long cg = a.c / vec, all = (long long)a.q.n_seq * cg;
    // Longer tiles read fewer rows twice and load the weights less often, shorter ones are more
    // threads.  Measured, bf16, 4 taps, us with 4, 8, 16, 32, 64 rows: 16384 x 4096 73, 59, 51.6, 50.9,
    // 51.8; 4096 x 4096 21.3, 18.3, 16.4, 15.8, 20.2; 1024 x 2048 4.1, 3.7, 4.3, 6.7, 10.9; 256 x 1024 2.9, 3.3,
    // 4.4, 6.6, 11.0.  No fewer rows than cached ones: only the first tile's window reaches those.
    const int least = a.k > 5 ? 8 : 4;
    auto tiles = [&](int rows) { return a.q.max_len / rows + (a.q.max_len % rows != 0); };
    const long long most = (long long)sms * 192;
    a.rows = 32;
    while (a.rows > least && all < most && all * tiles(a.rows) < most) a.rows /= 2;
    a.tiles = a.q.max_len ? tiles(a.rows) : 1;
    if (all > 0x7FFFFFFFLL * 128 / a.tiles) return cudaErrorInvalidConfiguration;
    a.threads = all * a.tiles;
    const long long blocks = (a.threads + 127) / 128;
    return launch(vec == VEC ? pick_conv<T, VEC>(a.k) : vec == 2 ? pick_conv<T, 2>(a.k) : pick_conv<T, 1>(a.k), dim3((unsigned)blocks), 128, 0, st, a);
}

}  // namespace seq
}  // namespace fcm

using namespace fcm;

extern "C" fcm_status fcm_causal_conv(const fcm_causal_conv_desc *desc, const void *x,
                                      const void *w, const float *s, const float *b,
                                      const void *state_in, void *y, void *state_out,
                                      void *stream) {
    FcmNvtxRange nvtx("fcm_causal_conv");
    if (!desc) return fcm_fail(FCM_ERR_INVALID_ARG, "desc is NULL");
    fcm_causal_conv_desc d = *desc;
    if (d.c < 1) return fcm_fail(FCM_ERR_INVALID_ARG, "c %d", d.c);
    if (d.ksize < 1 || d.ksize > seq::kMaxTaps)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "ksize %d outside 1..%d", d.ksize, seq::kMaxTaps);
    if (d.dtype < FCM_F32 || d.dtype > FCM_BF16)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "dtype %d: f32, f16 and bf16 are supported", d.dtype);
    if (d.act < FCM_ACT_NONE || d.act > FCM_ACT_SILU)
        return fcm_fail(FCM_ERR_INVALID_ARG, "activation code out of range");
    if (d.ksize == 1) state_in = state_out = nullptr;
    seq::ConvArgs a = {};
    fcm_status st;
    if ((st = seq::check_seqs(d.seqs, state_in || state_out, &a.q)) != FCM_OK ||
        (st = seq::check_ld(&d.ld_x, d.c, "ld_x")) != FCM_OK ||
        (st = seq::check_ld(&d.ld_y, d.c, "ld_y")) != FCM_OK)
        return st;
    if (a.q.n_seq == 0) return FCM_OK;
    const size_t e = (size_t)fcm_dtype_bytes(d.dtype);
    const bool rows = a.q.tokens > 0;   // x and y may be NULL when there is no row
    if ((rows && (st = seq::check_dev_ptr(x, e, "x")) != FCM_OK) ||
        (rows && (st = seq::check_dev_ptr(y, e, "y")) != FCM_OK) ||
        (st = seq::check_dev_ptr(w, e, "w")) != FCM_OK ||
        (s && (st = seq::check_dev_ptr(s, 4, "s")) != FCM_OK) ||
        (b && (st = seq::check_dev_ptr(b, 4, "b")) != FCM_OK) ||
        (state_in && (st = seq::check_dev_ptr(state_in, e, "state_in")) != FCM_OK) ||
        (state_out && (st = seq::check_dev_ptr(state_out, e, "state_out")) != FCM_OK))
        return st;
    if (seq::rows_overlap(x, d.ld_x, d.c, y, d.ld_y, d.c, a.q.tokens, e))
        return fcm_fail(FCM_ERR_INVALID_ARG, "x and y overlap");
    const long long state_row = (long long)(d.ksize - 1) * d.c;
    if (state_in != state_out &&
        seq::rows_overlap(state_in, state_row, state_row, state_out, state_row, state_row, a.q.slots, e))
        return fcm_fail(FCM_ERR_INVALID_ARG, "state_in and state_out overlap without being the same");
    int sms;
    if ((st = seq::current_device(&sms)) != FCM_OK) return st;

    a.x = x, a.w = w, a.s = s, a.b = b, a.state_in = state_in, a.y = y, a.state_out = state_out;
    a.ld_x = d.ld_x, a.ld_y = d.ld_y, a.c = d.c, a.k = d.ksize, a.act = d.act;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t ce = d.dtype == FCM_F32   ? seq::run_conv<float>(a, sms, cs)
                           : d.dtype == FCM_F16 ? seq::run_conv<__half>(a, sms, cs)
                                                : seq::run_conv<__nv_bfloat16>(a, sms, cs);
    if (ce != cudaSuccess) return fcm_fail(FCM_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(ce));
    return FCM_OK;
}
