// Attention over an 8-bit cache.
#include "kv_attend_kernel.cuh"

namespace graft {

cudaError_t prepare_kv_attend_eight() {
  const cudaError_t e = prepare_form<true, false>();
  return e != cudaSuccess ? e : prepare_form<true, true>();
}

cudaError_t launch_kv_attend_eight(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, int dtype, bool shaped, cudaStream_t s) {
  return shaped ? launch_form<true, true>(a, qmap, kmap, vmap, dtype, s) : launch_form<true, false>(a, qmap, kmap, vmap, dtype, s);
}

}  // namespace graft
