// Attention over the 8-bit cache, heads of 128.
#include "cache_attn.cuh"

namespace ibwd {

size_t cache_attention_workspace(int dim) {
  // a record a block, and two parts of up to 32 rows (16 of heads of 256)
  return kAttnGrid * (sizeof(JoinRecord) + 2 * (dim == 256 ? 16 : 32) * (size_t)part_row(dim) * sizeof(float));
}

cudaError_t cache_attention_128(const CacheAttnArgs& a, cudaStream_t st) { return attn_launch_of<128>(a, st); }

}  // namespace ibwd
