// Layer norm of fp16 rows.
#include "layer_norm.cuh"

namespace ibwd {

cudaError_t norm_fwd_f16(const NormFwdArgs& a, cudaStream_t st) { return norm_fwd<__half, __half>(a, st); }

cudaError_t norm_bwd_f16(const NormBwdArgs& a, cudaStream_t st) {
  return a.dy_type == 0 ? norm_bwd<__half, float>(a, st) : norm_bwd<__half, __half>(a, st);
}

}  // namespace ibwd
