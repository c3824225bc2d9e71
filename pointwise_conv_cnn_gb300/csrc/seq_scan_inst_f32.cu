// The selective scan's prompt kernel on f32 activations.
#include "seq_scan.cuh"

namespace fcm {
namespace seq {
FCM_SCAN_INSTANTIATE(float)
}  // namespace seq
}  // namespace fcm
