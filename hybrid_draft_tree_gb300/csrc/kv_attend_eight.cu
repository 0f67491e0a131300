// Attention over an 8-bit cache, plain scores.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendEightPlain = {prepare_form<true, kPlain>, launch_form<true, kPlain>};
}  // namespace graft
