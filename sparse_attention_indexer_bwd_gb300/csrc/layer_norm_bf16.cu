// Layer norm of bf16 rows.
#include "layer_norm.cuh"

namespace ibwd {

cudaError_t norm_fwd_bf16(const NormFwdArgs& a, cudaStream_t st) { return norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, st); }

cudaError_t norm_bwd_bf16(const NormBwdArgs& a, cudaStream_t st) {
  return a.dy_type == 0 ? norm_bwd<__nv_bfloat16, float>(a, st) : norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace ibwd
