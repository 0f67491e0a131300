// Arguments of the logit-rules kernel (logit_rules.cu), filled by api.cu.
#pragma once
#include "graft_internal.cuh"

namespace graft {

struct LogitArgs {
  graft_logit_rules r;
  int32_t V, batch, slots;
  const int32_t* tree_tok;
  const uint64_t* tree_mask;
  const void* in;
  void* out;
  int64_t in_stride, out_stride;
  int32_t chunk, rows_per_cta;  // set by the launcher: vocabulary of a CTA, slots of a CTA
  uint32_t* err;
};

cudaError_t prepare_logit_rules();  // once a device: the shared-memory opt-in
cudaError_t launch_logit_rules(const LogitArgs& a, int dtype, int num_sms, cudaStream_t s);

}  // namespace graft
