// Layer norm of fp32 rows.
#include "layer_norm.cuh"

namespace ibwd {

cudaError_t norm_fwd_f32(const NormFwdArgs& a, cudaStream_t st) {
  if (a.y_type == 0) return norm_fwd<float, float>(a, st);
  if (a.y_type == 1) return norm_fwd<float, __nv_bfloat16>(a, st);
  return norm_fwd<float, __half>(a, st);
}

cudaError_t norm_bwd_f32(const NormBwdArgs& a, cudaStream_t st) {
  if (a.dy_type == 0) return norm_bwd<float, float>(a, st);
  if (a.dy_type == 1) return norm_bwd<float, __nv_bfloat16>(a, st);
  return norm_bwd<float, __half>(a, st);
}

}  // namespace ibwd
