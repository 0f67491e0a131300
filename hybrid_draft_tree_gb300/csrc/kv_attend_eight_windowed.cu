// Attention over an 8-bit cache, scores inside a window.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendEightWindowed = {prepare_form<true, kWindowed>, launch_form<true, kWindowed>};
}  // namespace graft
