// Norm and rotation of heads in bf16.
#include "head_norm.cuh"

namespace ibwd {

cudaError_t heads_bf16(const HeadArgs& a, bool backward, cudaStream_t st) {
  return backward ? launch_heads_of<__nv_bfloat16, true>(a, st) : launch_heads_of<__nv_bfloat16, false>(a, st);
}

}  // namespace ibwd
