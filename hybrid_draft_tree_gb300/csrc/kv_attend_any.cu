// Attention over a cache in the model's type, capped scores that fall with the distance, and caps of any size.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendAny = {prepare_form<false, kAny>, launch_form<false, kAny>};
}  // namespace graft
