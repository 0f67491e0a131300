// Attention with capped, windowed or distance-biased scores over a cache in the model's type.
#include "kv_attend_kernel.cuh"

namespace graft {

cudaError_t prepare_kv_attend_shaped() { return prepare_form<false, true>(); }

cudaError_t launch_kv_attend_shaped(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                    const CUtensorMap& vmap, int dtype, cudaStream_t s) {
  return launch_form<false, true>(a, qmap, kmap, vmap, dtype, s);
}

}  // namespace graft
