// Norm and rotation of heads in fp16.
#include "head_norm.cuh"

namespace ibwd {

cudaError_t heads_f16(const HeadArgs& a, bool backward, cudaStream_t st) {
  return backward ? launch_heads_of<__half, true>(a, st) : launch_heads_of<__half, false>(a, st);
}

}  // namespace ibwd
