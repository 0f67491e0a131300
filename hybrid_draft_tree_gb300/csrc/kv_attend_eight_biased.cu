// Attention over an 8-bit cache, scores that fall with the distance.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendEightBiased = {prepare_form<true, kBiased>, launch_form<true, kBiased>};
}  // namespace graft
