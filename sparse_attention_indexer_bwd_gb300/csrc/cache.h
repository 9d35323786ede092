// Launchers of the 8-bit cache (cache.cu) and of the attention over it
// (cache_attn.cuh), shared with cache_api.cu.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ibwd {

// Sequences whose tokens lie in pages.
struct CacheSeqs {
  const int32_t* table;  // [batch, width] page numbers, `stride` elements apart
  const int32_t* lens;   // [batch]
  const int32_t* cu;     // [batch + 1] or nullptr: one token a sequence
  long long stride, pages, tokens;
  int batch, width;
  int page_log;  // log2 of a page's tokens

  // Tokens of sequence b that the pages can hold.
  __device__ int length(int b) const {
    const int len = lens[b];
    const long long most = (long long)width << page_log;
    return len < 0 ? 0 : len > most ? (int)most : len;
  }
  // The packed tokens of sequence b begin at begin(b) and end before begin(b + 1).
  __device__ int begin(int b) const {
    if (!cu) return b;
    const int v = cu[b];
    return v < 0 ? 0 : v > tokens ? (int)tokens : v;
  }
  // The page that holds position `at` of sequence b; -1 where there is none.
  __device__ int page_at(int b, int at) const {
    const int p = table[b * stride + (at >> page_log)];
    return p < 0 || p >= pages ? -1 : p;
  }
};

struct CacheWriteArgs {
  const void* x[2];  // keys, values: [tokens, heads, dim]
  long long token[2], head[2];
  void* codes[2];  // [pages, heads, page, dim]
  float* scale[2];  // [pages, heads]
  CacheSeqs seqs;
  int type, code, heads, dim;
};
cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t st);

struct CacheReadArgs {
  const void* codes;
  const float* scale;
  void* out;  // [batch, length, heads, dim]
  CacheSeqs seqs;
  int type, code, heads, dim, length;
};
cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t st);

struct CacheAttnArgs {
  const void* q;  // [tokens, heads * group, dim]
  long long q_token, q_head;
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  CacheSeqs seqs;
  const int32_t* select;  // [tokens, kept] or nullptr
  int kept;
  void* out;   // as q, contiguous
  float* lse;  // [tokens, heads * group] or nullptr
  int type, code, heads, group, dim;
  float scale_log2;  // of a logit, in base-2 logarithms
  void* work;
  int num_sms;
};
size_t cache_attention_workspace(int dim);
cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st);
// The same by head width.
cudaError_t cache_attention_64(const CacheAttnArgs& a, cudaStream_t st);
cudaError_t cache_attention_128(const CacheAttnArgs& a, cudaStream_t st);
cudaError_t cache_attention_256(const CacheAttnArgs& a, cudaStream_t st);

}  // namespace ibwd
