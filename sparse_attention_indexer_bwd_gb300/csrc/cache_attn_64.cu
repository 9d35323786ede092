// Attention over the 8-bit cache, heads of 64.
#include "cache_attn.cuh"

namespace ibwd {

cudaError_t cache_attention_64(const CacheAttnArgs& a, cudaStream_t st) { return attn_launch_of<64>(a, st); }

}  // namespace ibwd
