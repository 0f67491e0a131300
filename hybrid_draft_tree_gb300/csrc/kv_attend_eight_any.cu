// Attention over an 8-bit cache, capped scores that fall with the distance, and caps of any size.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendEightAny = {prepare_form<true, kAny>, launch_form<true, kAny>};
}  // namespace graft
