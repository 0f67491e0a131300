// Attention over a cache in the model's type, scores that fall with the distance.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendBiased = {prepare_form<false, kBiased>, launch_form<false, kBiased>};
}  // namespace graft
