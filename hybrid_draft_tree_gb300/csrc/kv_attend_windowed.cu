// Attention over a cache in the model's type, scores inside a window.
#include "kv_attend_kernel.cuh"

namespace graft {
const AttendForm kAttendWindowed = {prepare_form<false, kWindowed>, launch_form<false, kWindowed>};
}  // namespace graft
