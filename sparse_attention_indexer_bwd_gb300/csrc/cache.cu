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

#include <cstring>
#include <type_traits>

#include "cache.h"
#include "elem.cuh"
#include "indexer_cache.h"
#include "kcommon.cuh"

namespace ibwd {

namespace {

constexpr int kWriteThreads = 128;
constexpr int kReadThreads = 128;
constexpr int kReadAhead = 8;  // loads in flight a thread

// Eight elements as they lie in memory; `vec`: on 16 bytes.
template <typename T>
struct Chunk {
  static constexpr uint32_t kInfinity = std::is_same<T, float>::value ? 0x7F800000u : std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  // A magnitude's bits as fp32's.
  __device__ static uint32_t bits_of(uint32_t m) {
    if constexpr (std::is_same<T, float>::value) return m;
    if constexpr (std::is_same<T, __half>::value) return __float_as_uint(unpack2(m, __half{}).x);
    return m << 16;
  }
  uint4 w[sizeof(T) / 2];
  __device__ void load(const T* p, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = *(reinterpret_cast<const uint4*>(p) + i);
    } else {
      T v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i];
      memcpy(w, v, sizeof(w));
    }
  }
  // The largest magnitude, as its type's bits (which are in their values' order; infinities and NaN above all): of 16-bit
  // elements in each half.
  __device__ uint32_t most(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = sizeof(T) == 2 ? __vmaxu2(m, x[j] & 0x7FFF7FFFu) : max(m, x[j] & 0x7FFFFFFFu);
    }
    return m;
  }
  __device__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
      unpack(w[0], v, T{});
    } else {
      float a[4], b[4];
      unpack(w[0], a, 0.f);
      unpack(w[1], b, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    }
  }
};

// The least power of two 2^e, e in [-126, 120], with amax <= M 2^e; amax finite. 120 is what the largest float needs in e4m3;
// whole numbers would need 122, at which their largest codes are no floats: what is beyond 127 * 2^120 gets the largest code.
template <bool INT8>
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127;                      // amax = 1.m 2^e
  const uint32_t most = INT8 ? 0x7E0000u : 0x600000u;         // the mantissa of 127 and of 448
  int s = e - (INT8 ? 6 : 8) + ((bits & 0x7FFFFFu) > most);
  s = bits < 0x800000u ? -126 : max(-126, min(120, s));
  return __uint_as_float((uint32_t)(s + 127) << 23);
}

// Four values in units of the scale to codes. int8: `tame` where all are numbers of at most 127, which the sum with
// 1.5 2^23 rounds into its lowest byte; else they are limited, and NaN becomes 0.
template <bool INT8>
__device__ __forceinline__ uint32_t code4(float4 v, bool tame) {
  if constexpr (INT8) {
    if (!tame) {
      auto limited = [](float f) { return f == f ? fminf(fmaxf(f, -127.f), 127.f) : 0.f; };
      v = make_float4(limited(v.x), limited(v.y), limited(v.z), limited(v.w));
    }
    auto byte = [](float f) { return __float_as_uint(f + 12582912.f); };
    return __byte_perm(__byte_perm(byte(v.x), byte(v.y), 0x0040), __byte_perm(byte(v.z), byte(v.w), 0x0040), 0x5410);
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.z, v.w), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
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
// HOLD of a thread's chunks stay in registers between the block's largest value
// and its codes: eight (four in fp32) are all of a page of 64 tokens of 128
// 16-bit elements, one is all of a few tokens a sequence, whose blocks are
// many and short (128 sequences, 8 heads: 6.8 us with eight, 4.7 with one).
// Others are read twice.
template <typename T, bool INT8, int HOLD>
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const __grid_constant__ CacheWriteArgs a, bool vec) {
  __shared__ uint32_t warp_max[kWriteThreads / 32];
  chained();
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

  const T* x0 = x + (from + (base + s0 - start)) * a.token[kv];  // the first slot's
  const int count = (s1 - s0) * chunks;
  // This thread's chunks: slot and place in it, without a division each.
  const int slots = kWriteThreads / chunks, places = kWriteThreads % chunks;
  const int slot0 = threadIdx.x / chunks, c0 = threadIdx.x - slot0 * chunks;
  auto onward = [&](int& slot, int& c) {
    slot += slots;
    c += places;
    if (c >= chunks) {
      c -= chunks;
      ++slot;
    }
  };
  Chunk<T> held[HOLD];
  int slot = slot0, c = c0;
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    if (threadIdx.x + k * kWriteThreads < count) held[k].load(x0 + slot * a.token[kv] + 8 * c, vec);
    onward(slot, c);
  }
  const int slot_on = slot, c_on = c;
  // f of every chunk of this thread
  auto every = [&](auto f) {
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (threadIdx.x + k * kWriteThreads < count) f(held[k], threadIdx.x + k * kWriteThreads);
    slot = slot_on;
    c = c_on;
    for (int i = threadIdx.x + HOLD * kWriteThreads; i < count; i += kWriteThreads) {
      Chunk<T> w;
      w.load(x0 + slot * a.token[kv] + 8 * c, vec);
      f(w, i);
      onward(slot, c);
    }
  };
  auto block_max = [&](uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWriteThreads / 32; ++w) v = max(v, warp_max[w]);
    return v;
  };
  uint32_t m = 0;
  every([&](const Chunk<T>& w, int) { m = w.most(m); });
  if (sizeof(T) == 2) m = max(m & 0xFFFFu, m >> 16);
  m = block_max(m);
  unsigned flags = 0;  // 1: there are infinities or NaN, 2: NaN in whole numbers
  if (m < Chunk<T>::kInfinity) {
    m = Chunk<T>::bits_of(m);
  } else {  // the largest of the finite ones then
    flags = 1u;
    uint32_t finite = 0, nan = 0;
    every([&](const Chunk<T>& w, int) {
      float v[8];
      w.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        finite = max(finite, x < 0x7F800000u ? x : 0u);
        nan |= x > 0x7F800000u;
      }
    });
    m = block_max(finite);
    if (INT8 && block_max(nan)) flags |= 2u;
  }
  const float need = scale_for<INT8>(__uint_as_float(m));
  const float kept = s0 ? fmaxf(old, need) : need;

  if (s0 && old != kept) {
    const float f = old / kept;
    for (int i = threadIdx.x; i < s0 * chunks; i += kWriteThreads) {
      const uint2 w = codes[i];
      float4 u = value4(w.x, INT8), v = value4(w.y, INT8);
      u.x *= f, u.y *= f, u.z *= f, u.w *= f;
      v.x *= f, v.y *= f, v.z *= f, v.w *= f;
      codes[i] = make_uint2(code4<INT8>(u, false), code4<INT8>(v, false));
    }
  }
  // a power of two has an exact inverse; a scale that someone else made is divided by
  const bool exact = (__float_as_uint(kept) & 0x7FFFFFu) == 0;
  const float inv = 1.f / kept;
  const bool tame = !flags && __uint_as_float(m) <= 127.f * kept;
  auto put = [&](const Chunk<T>& w, int i) {
    float v[8];
    w.get(v);
    if (exact) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= inv;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] /= kept;
    }
    codes[s0 * chunks + i] = make_uint2(code4<INT8>(make_float4(v[0], v[1], v[2], v[3]), tame),
                                        code4<INT8>(make_float4(v[4], v[5], v[6], v[7]), tame));
  };
  every(put);
  // whole numbers have no NaN: the block's scale is one instead, and stays it
  if (threadIdx.x == 0) *scale = INT8 && (flags & 2u || old != old) ? __uint_as_float(0x7FC00000u) : kept;
}

// As many codes a lane as make 16 bytes of the result, in the cache's order: a
// warp's reads and writes are runs of whole sectors. x: a sequence's page, y: a head.
// LANES: the threads that share a page, a warp where it has up to 4096 codes
// (8x8192x8 tokens of 64 in pages of 16: 20 us, a block a page 36).
template <typename T, bool INT8, int LANES>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ CacheReadArgs a, int pages) {
  chained();
  const CacheSeqs& s = a.seqs;
  const long long at = (long long)blockIdx.x * (kReadThreads / LANES) + threadIdx.x / LANES;
  const int b = (int)(at / pages), index = (int)(at - (long long)b * pages), head = blockIdx.y, P = 1 << s.page_log;
  if (b >= s.batch) return;
  const int base = index << s.page_log, rows = min(P, a.length - base);
  const int len = s.length(b);
  const int page = base < len ? s.page_at(b, base) : -1;
  const long long block = (long long)page * a.heads + head;
  const float scale = page >= 0 ? a.scale[block] : 0.f;
  constexpr int V = 16 / sizeof(T);  // codes
  using Codes = typename std::conditional<V == 8, uint2, uint32_t>::type;
  const Codes* codes = reinterpret_cast<const Codes*>(static_cast<const uint8_t*>(a.codes) + block * P * a.dim);
  const int chunks = a.dim / V;
  const int total = rows * chunks, held = page < 0 ? 0 : min(rows, len - base) * chunks;
  for (int i0 = threadIdx.x % LANES; i0 < total; i0 += kReadAhead * LANES) {
    Codes r[kReadAhead];
#pragma unroll
    for (int k = 0; k < kReadAhead; ++k) {
      const int i = i0 + k * LANES;
      r[k] = Codes{};
      if (i < held) r[k] = __ldcs(codes + i);
    }
#pragma unroll
    for (int k = 0; k < kReadAhead; ++k) {
      const int i = i0 + k * LANES, slot = i / chunks, c = i - slot * chunks;
      if (i >= total) break;
      T* out = static_cast<T*>(a.out) + (((long long)b * a.length + base + slot) * a.heads + head) * a.dim + V * c;
      const float by = i < held ? scale : 0.f;  // (behind the end even where the scale is no number)
      auto scaled = [&](uint32_t w) {
        const float4 v = value4(w, INT8);
        return make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
      };
      if constexpr (V == 8) {
        const float4 v = scaled(r[k].x), w = scaled(r[k].y);
        st_stream(out, make_uint4(pack2_of(make_float2(v.x, v.y), T{}), pack2_of(make_float2(v.z, v.w), T{}),
                                  pack2_of(make_float2(w.x, w.y), T{}), pack2_of(make_float2(w.z, w.w), T{})));
      } else {
        const float4 v = scaled(r[k]);
        st_stream(out, make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)));
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
    constexpr int kMost = sizeof(T) == 2 ? 8 : 4;
    auto go = [&](auto kern) { return launch_ex(kern, grid, kWriteThreads, 0, st, true, a, vec); };
    const bool few = s.tokens * (a.dim / 8) <= (long long)kWriteThreads * s.batch;
    if (a.code == IBWD_INT8) return few ? go(write_kernel<T, true, 1>) : go(write_kernel<T, true, kMost>);
    return few ? go(write_kernel<T, false, 1>) : go(write_kernel<T, false, kMost>);
  });
}

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t st) {
  const int P = 1 << a.seqs.page_log, pages = (a.length + P - 1) / P;
  const bool small = P * a.dim <= 4096;
  const long long blocks = small ? ((long long)pages * a.seqs.batch + kReadThreads / 32 - 1) / (kReadThreads / 32)
                                 : (long long)pages * a.seqs.batch;
  const dim3 grid((unsigned)blocks, a.heads);
  return by_type(a.type, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto kern) { return launch_ex(kern, grid, kReadThreads, 0, st, true, a, pages); };
    if (a.code == IBWD_INT8) return small ? go(read_kernel<T, true, 32>) : go(read_kernel<T, true, kReadThreads>);
    return small ? go(read_kernel<T, false, 32>) : go(read_kernel<T, false, kReadThreads>);
  });
}

}  // namespace ibwd
