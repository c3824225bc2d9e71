// seq_common.cu -- host checks shared by the layers over sequences.
#include "seq_common.cuh"

#include <atomic>

namespace fcm {
namespace seq {

fcm_status check_seqs(const fcm_seqs &s, bool state, Seqs *out) {
    if (s.n_seq < 0 || s.max_len < 0 || s.tokens < 0)
        return fcm_fail(FCM_ERR_INVALID_ARG, "negative tokens, n_seq or max_len");
    if (s.tokens > (1LL << 31) - 1)
        return fcm_fail(FCM_ERR_UNSUPPORTED, "%lld tokens; at most 2^31 - 1", s.tokens);
    if (s.n_seq > 1 << 30) return fcm_fail(FCM_ERR_UNSUPPORTED, "%d sequences; at most 2^30", s.n_seq);
    if (!s.seq_start && s.tokens != (long long)s.n_seq * s.max_len)
        return fcm_fail(FCM_ERR_INVALID_ARG,
                        "%lld tokens are not n_seq %d times max_len %d (no seq_start)", s.tokens,
                        s.n_seq, s.max_len);
    if (state && s.slots < 1 && s.n_seq > 0)
        return fcm_fail(FCM_ERR_INVALID_ARG, "a state was given, but slots is %d", s.slots);
    if (state && !s.slot && s.slots < s.n_seq)
        return fcm_fail(FCM_ERR_INVALID_ARG, "%d slots hold no state for each of %d sequences",
                        s.slots, s.n_seq);
    if (reinterpret_cast<uintptr_t>(s.seq_start) % 4 || reinterpret_cast<uintptr_t>(s.slot) % 4)
        return fcm_fail(FCM_ERR_ALIGNMENT, "seq_start or slot is not 4-byte aligned");
    out->seq_start = s.seq_start;
    out->slot = s.slot;
    out->tokens = s.tokens;
    out->n_seq = s.n_seq;
    // a bound of the lengths that is past all tokens says no more than the tokens do
    out->max_len = s.seq_start && s.max_len > s.tokens ? (int)s.tokens : s.max_len;
    out->slots = s.slots;
    return FCM_OK;
}

fcm_status check_ld(long long *ld, long long row, const char *name) {
    if (*ld == 0) *ld = row;
    if (*ld < row || *ld > 0x7FFFFFFFLL)
        return fcm_fail(FCM_ERR_INVALID_ARG, "%s %lld: rows of %lld elements need at least that, "
                        "and at most 2^31 - 1", name, *ld, row);
    return FCM_OK;
}

fcm_status check_dev_ptr(const void *p, size_t align, const char *name) {
    if (!p) return fcm_fail(FCM_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align)
        return fcm_fail(FCM_ERR_ALIGNMENT, "%s is not %zu-byte aligned", name, align);
    return FCM_OK;
}

bool rows_overlap(const void *a, long long lda, long long ca, const void *b, long long ldb,
                  long long cb, long long rows, size_t esize) {
    if (!a || !b || rows <= 0 || ca <= 0 || cb <= 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    const uintptr_t na = (uintptr_t)((rows - 1) * lda + ca) * esize;
    const uintptr_t nb = (uintptr_t)((rows - 1) * ldb + cb) * esize;
    if (pa >= pb + nb || pb >= pa + na) return false;
    if (lda != ldb) return true;
    const long long ld = lda * (long long)esize, wa = ca * (long long)esize, wb = cb * (long long)esize;
    long long off = pb >= pa ? (long long)((pb - pa) % (uintptr_t)ld)
                             : (ld - (long long)((pa - pb) % (uintptr_t)ld)) % ld;
    return off < wa || off + wb > ld;   // b's columns start inside a's, or run into a's next row
}

fcm_status current_device(int *num_sms) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> sms[kMaxDevices];   // 0: not looked at yet, -1: not a 10.3 device
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
        cudaGetLastError();
        return fcm_fail(FCM_ERR_NO_DEVICE, "no CUDA device");
    }
    int n = dev < kMaxDevices ? sms[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        int major = 0, minor = 0;
        cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fcm_fail(FCM_ERR_NO_DEVICE, "no CUDA device: %s", cudaGetErrorString(e));
        }
        if (major != 10 || minor != 3) n = -1;
        if (dev < kMaxDevices) sms[dev].store(n, std::memory_order_relaxed);
    }
    if (n < 0)
        return fcm_fail(FCM_ERR_NO_DEVICE,
                        "device %d is not compute capability 10.3; this library is built for sm_103a",
                        dev);
    *num_sms = n;
    return FCM_OK;
}

}  // namespace seq
}  // namespace fcm
