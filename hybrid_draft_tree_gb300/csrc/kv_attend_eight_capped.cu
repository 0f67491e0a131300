// Attention over an 8-bit cache, capped scores.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendEightCapped = {prepare_form<true, kCapped>, launch_form<true, kCapped>};
}  // namespace graft
