// Norm and rotation of heads in fp32.
#include "head_norm.cuh"

namespace ibwd {

cudaError_t heads_f32(const HeadArgs& a, bool backward, cudaStream_t st) {
  return backward ? launch_heads_of<float, true>(a, st) : launch_heads_of<float, false>(a, st);
}

}  // namespace ibwd
