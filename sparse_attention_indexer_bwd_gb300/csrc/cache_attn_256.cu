// Attention over the 8-bit cache, heads of 256.
#include "cache_attn.cuh"

namespace ibwd {

cudaError_t cache_attention_256(const CacheAttnArgs& a, cudaStream_t st) { return attn_launch_of<256>(a, st); }

}  // namespace ibwd
