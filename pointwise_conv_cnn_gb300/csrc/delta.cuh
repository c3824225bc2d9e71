// delta.cuh -- what the gated delta rule's kernels share.
#pragma once

#include "seq_common.cuh"
#include "tc_common.cuh"

namespace fcm {
namespace seq {

constexpr int kMaxDeltaKeys = 256;
constexpr int kDeltaCols = 32;        // value columns of a block
constexpr float kDeltaEps = 1e-6f;    // beside a key's sum of squares

struct DeltaArgs {
    Seqs q;
    const void *qp, *kp, *vp, *dt, *b;
    const float *a, *dt_bias, *state_in;
    void *y;
    float *state_out;
    long long ld_q, ld_k, ld_v, ld_dt, ld_b, ld_y;
    int heads, per_key, dk, dv;   // per_key: heads of one key head
    int slices;                   // blocks of columns
    int softplus, sigmoid, normalize;
    float scale;
    int vec, vec_v;   // eight keys and queries, values, of a row may be read at once
};

// G of one row and head, and its step B.  A scalar a row: the library's functions, whose errors are units of
// the last place.
__device__ __forceinline__ float log_decay(float v, float a, int softplus) {
    if (softplus) v = (v < 0.0f ? 0.0f : v) + log1pf(expf(-fabsf(v)));
    return v * a;
}
__device__ __forceinline__ float step_of(float v, int sigmoid) { return sigmoid ? 1.0f / (1.0f + expf(-v)) : v; }

}  // namespace seq
}  // namespace fcm
