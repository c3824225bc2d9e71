// The selective scan's prompt kernel on bf16 activations.
#include "seq_scan.cuh"

namespace fcm {
namespace seq {
FCM_SCAN_INSTANTIATE(__nv_bfloat16)
}  // namespace seq
}  // namespace fcm
