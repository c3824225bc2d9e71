// The selective scan's prompt kernel on f16 activations.
#include "seq_scan.cuh"

namespace fcm {
namespace seq {
FCM_SCAN_INSTANTIATE(__half)
}  // namespace seq
}  // namespace fcm
