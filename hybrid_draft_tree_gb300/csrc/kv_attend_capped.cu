// Attention over a cache in the model's type, capped scores.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendCapped = {prepare_form<false, kCapped>, launch_form<false, kCapped>};
}  // namespace graft
