// Writing a paged 8-bit cache, and reading it back.
//
// A block of the cache is one head's tokens of one page; its codes stand for
// code * scale. The scale is a power of two, the least at which nothing finite
// that the block was given is beyond the largest code M (448 in e4m3, 127 in
// whole numbers): x / scale is exact, so a code has one rounding, and where a
// later token raises the scale the older codes move by an exact factor (e4m3
// codes keep their value but for those that fall below its normal range; whole
// numbers lose half a unit of the new scale). Scales of M / amax would round
// twice, and again at every token that raises them.
#include <cuda_fp8.h>

#include "cache.h"
#include "elem.cuh"
#include "indexer_cache.h"
#include "kcommon.cuh"

namespace ibwd {

namespace {

constexpr int kWriteThreads = 128;
constexpr int kReadThreads = 128;
constexpr int kReadAhead = 4;  // 16-byte loads in flight a thread

template <typename T>
__device__ __forceinline__ void load_some(const T* p, float (&v)[8], bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      unpack(*reinterpret_cast<const uint4*>(p), v, T{});
    } else {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
  }
}

// The least power of two 2^e, e in [-126, 120], with amax <= M 2^e; amax finite.
template <bool INT8>
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127;                      // amax = 1.m 2^e
  const uint32_t most = INT8 ? 0x7E0000u : 0x600000u;         // the mantissa of 127 and of 448
  int s = e - (INT8 ? 6 : 8) + ((bits & 0x7FFFFFu) > most);
  s = bits < 0x800000u ? -126 : max(-126, min(120, s));
  return __uint_as_float((uint32_t)(s + 127) << 23);
}

__device__ __forceinline__ uint32_t code4(float4 v, bool int8) {
  if (int8) {
    // (NaN becomes 0)
    auto one = [](float f) { return (uint32_t)(__float2int_rn(fminf(fmaxf(f, -127.f), 127.f)) & 0xFF); };
    auto num = [&](float f) { return f == f ? one(f) : 0u; };
    return num(v.x) | num(v.y) << 8 | num(v.z) << 16 | num(v.w) << 24;
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.z, v.w), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

__device__ __forceinline__ float4 value4(uint32_t c, bool int8) {
  if (int8)
    return make_float4((float)(int8_t)(c & 0xFF), (float)(int8_t)(c >> 8 & 0xFF), (float)(int8_t)(c >> 16 & 0xFF),
                       (float)(int8_t)(c >> 24));
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFF), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// The largest b in [0, n) with first(b) <= x, for first() that does not fall;
// 32 places at a time, by a warp.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, long long x, F first) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (int)(threadIdx.x & 31) * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && (at == lo || first(at) <= x));
    const int run = __popc(below) - 1;
    lo += run * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// One block of the cache a block of threads: blockIdx.x is the x-th of at most
// tokens / page + 2 batch pieces (a sequence's n new tokens touch at most
// n / page + 2 pages), y the head, z keys or values.
template <typename T, bool INT8>
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const __grid_constant__ CacheWriteArgs a, bool vec) {
  __shared__ uint32_t warp_max[kWriteThreads / 32];
  const CacheSeqs& s = a.seqs;
  const int head = blockIdx.y, kv = blockIdx.z, P = 1 << s.page_log;
  int b = blockIdx.x, piece = 0;
  if (s.cu) {
    auto first = [&](int i) { return (long long)(s.begin(i) >> s.page_log) + 2ll * i; };
    b = last_at_most(s.batch, blockIdx.x, first);
    piece = (int)(blockIdx.x - first(b));
  }
  const int from = s.begin(b), n = s.begin(b + 1) - from, len = s.length(b);
  // (a length beyond the pages is cut there, its last tokens with it)
  const long long start = (long long)max(s.lens[b], 0) - n;
  const int p0 = (int)max(start, 0ll);
  const long long page_index = (long long)(p0 >> s.page_log) + piece;
  if (n <= 0 || piece < 0 || p0 >= len || page_index > (len - 1) >> s.page_log) return;
  const int page = s.page_at(b, (int)(page_index << s.page_log));
  if (page < 0) return;
  const int base = (int)(page_index << s.page_log);
  const int s0 = max(p0, base) - base, s1 = min(len, base + P) - base;
  const int chunks = a.dim >> 3;
  const T* x = static_cast<const T*>(a.x[kv]) + head * a.head[kv];
  const long long block = (long long)page * a.heads + head;
  uint2* codes = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.codes[kv]) + block * P * a.dim);
  float* scale = a.scale[kv] + block;
  const float old = s0 ? *scale : 0.f;

  auto row = [&](int slot) { return x + (from + (base + slot - start)) * a.token[kv]; };
  uint32_t most = 0;  // bits of the largest finite |x|; the highest bit: there is a NaN
  for (int i = threadIdx.x; i < (s1 - s0) * chunks; i += kWriteThreads) {
    const int slot = s0 + i / chunks, c = i % chunks;
    float v[8];
    load_some(row(slot) + 8 * c, v, vec);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = __float_as_uint(v[j]) & 0x7FFFFFFFu;
      if (m < 0x7F800000u)
        most = max(most, m);
      else if (INT8 && m > 0x7F800000u)
        most |= 0x80000000u;
    }
  }
  {
    const bool nan = __any_sync(0xffffffffu, most >> 31);
    uint32_t m = __reduce_max_sync(0xffffffffu, most & 0x7FFFFFFFu);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m | (nan ? 0x80000000u : 0u);
  }
  __syncthreads();
  uint32_t m = 0, nan = 0;
#pragma unroll
  for (int w = 0; w < kWriteThreads / 32; ++w) {
    m = max(m, warp_max[w] & 0x7FFFFFFFu);
    nan |= warp_max[w] >> 31;
  }
  const float need = scale_for<INT8>(__uint_as_float(m));
  const float kept = s0 ? fmaxf(old, need) : need;

  if (s0 && old != kept) {
    const float f = old / kept;
    for (int i = threadIdx.x; i < s0 * chunks; i += kWriteThreads) {
      uint2 c = codes[i];
      float4 u = value4(c.x, INT8), w = value4(c.y, INT8);
      u.x *= f, u.y *= f, u.z *= f, u.w *= f;
      w.x *= f, w.y *= f, w.z *= f, w.w *= f;
      codes[i] = make_uint2(code4(u, INT8), code4(w, INT8));
    }
  }
  // a power of two has an exact inverse; a scale that someone else made is divided by
  const bool exact = (__float_as_uint(kept) & 0x7FFFFFu) == 0;
  const float inv = 1.f / kept;
  for (int i = threadIdx.x; i < (s1 - s0) * chunks; i += kWriteThreads) {
    const int slot = s0 + i / chunks, c = i % chunks;
    float v[8];
    load_some(row(slot) + 8 * c, v, vec);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = exact ? v[j] * inv : v[j] / kept;
    codes[slot * chunks + c] = make_uint2(code4(make_float4(v[0], v[1], v[2], v[3]), INT8),
                                          code4(make_float4(v[4], v[5], v[6], v[7]), INT8));
  }
  // whole numbers have no NaN: the block's scale is one instead, and stays it
  if (threadIdx.x == 0) *scale = INT8 && (nan || old != old) ? __uint_as_float(0x7FC00000u) : kept;
}

// Sixteen codes a thread, in the cache's order: a warp's reads are one run of
// 512 bytes. x: a sequence's page, y: a head.
template <typename T, bool INT8>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ CacheReadArgs a, int pages) {
  const CacheSeqs& s = a.seqs;
  const int b = blockIdx.x / pages, index = blockIdx.x - b * pages, head = blockIdx.y, P = 1 << s.page_log;
  const int base = index << s.page_log, rows = min(P, a.length - base);
  const int len = s.length(b);
  const int page = base < len ? s.page_at(b, base) : -1;
  const long long block = (long long)page * a.heads + head;
  const float scale = page >= 0 ? a.scale[block] : 0.f;
  const uint4* codes = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.codes) + block * P * a.dim);
  const int chunks = a.dim >> 4;
  const int total = rows * chunks, held = page < 0 ? 0 : min(rows, len - base) * chunks;
  for (int i0 = threadIdx.x; i0 < total; i0 += kReadAhead * kReadThreads) {
    uint4 r[kReadAhead];
#pragma unroll
    for (int k = 0; k < kReadAhead; ++k) {
      const int i = i0 + k * kReadThreads;
      r[k] = i < held ? ld_stream(codes + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kReadAhead; ++k) {
      const int i = i0 + k * kReadThreads, slot = i / chunks, c = i - slot * chunks;
      if (i >= total) break;
      T* out = static_cast<T*>(a.out) + (((long long)b * a.length + base + slot) * a.heads + head) * a.dim + 16 * c;
      const uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
      const float by = i < held ? scale : 0.f;  // (behind the end even where the scale is no number)
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = value4(w[j], INT8);
        v[j].x *= by, v[j].y *= by, v[j].z *= by, v[j].w *= by;
      }
      if constexpr (sizeof(T) == 2) {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[2 * j] = pack2_of(make_float2(v[j].x, v[j].y), T{});
          h[2 * j + 1] = pack2_of(make_float2(v[j].z, v[j].w), T{});
        }
        st_stream(out, make_uint4(h[0], h[1], h[2], h[3]));
        st_stream(out + 8, make_uint4(h[4], h[5], h[6], h[7]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_stream(out + 4 * j, make_uint4(__float_as_uint(v[j].x), __float_as_uint(v[j].y), __float_as_uint(v[j].z),
                                            __float_as_uint(v[j].w)));
      }
    }
  }
}

// f of a value of the element type.
template <typename F>
cudaError_t by_type(int type, F f) {
  if (type == IBWD_F32) return f(float{});
  if (type == IBWD_BF16) return f(__nv_bfloat16{});
  return f(__half{});
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t st) {
  const CacheSeqs& s = a.seqs;
  const int size = a.type == IBWD_F32 ? 4 : 2, kinds = a.x[1] ? 2 : 1;
  bool vec = true;
  for (int i = 0; i < kinds; ++i)
    vec = vec && reinterpret_cast<uintptr_t>(a.x[i]) % 16 == 0 && a.token[i] * size % 16 == 0 && a.head[i] * size % 16 == 0;
  const long long pieces = s.cu ? (s.tokens >> s.page_log) + 2ll * s.batch : s.batch;
  const dim3 grid((unsigned)pieces, a.heads, kinds);
  return by_type(a.type, [&](auto t) {
    using T = decltype(t);
    return launch_ex(a.code == IBWD_INT8 ? write_kernel<T, true> : write_kernel<T, false>, grid, kWriteThreads, 0, st, false, a,
                     vec);
  });
}

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t st) {
  const int P = 1 << a.seqs.page_log, pages = (a.length + P - 1) / P;
  const dim3 grid((unsigned)((long long)pages * a.seqs.batch), a.heads);
  return by_type(a.type, [&](auto t) {
    using T = decltype(t);
    return launch_ex(a.code == IBWD_INT8 ? read_kernel<T, true> : read_kernel<T, false>, grid, kReadThreads, 0, st, false, a,
                     pages);
  });
}

}  // namespace ibwd
