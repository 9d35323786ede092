// What the kernels over rows of logits share: a block's part of a row, and
// the running statistic (maximum, sum of exponentials, their first moment).
#pragma once
#include "elem.cuh"
#include "packed.cuh"
#include "ptx.cuh"
#include "train.h"

namespace ibwd {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;  // vectors a thread takes together
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
// An exponent whose power of two is 0, kept finite so that 0 times it is 0.
constexpr float kLeast = -1e20f;
// The largest of a teacher's weights, of which there are 1024 at most, so that
// the loss's sums over tokens at the type's lowest value stay in range.
constexpr float kShare = 1.f / 2048.f;
constexpr float kLargest = 3.40282347e38f;
#define NEG_INF (-INFINITY)

struct Stat {
  float m, s, u;
};

// The reference point of the exponents: the maximum, or 0 while there is none
// (every term is then 2^-inf = 0; x - m of two infinities never occurs).
__device__ __forceinline__ float finite_max(float m) { return m == NEG_INF ? 0.f : m; }

// The part [lo, hi) of a row as a block reads it: single elements up to a
// 16-byte boundary, whole 16-byte vectors, single elements.
template <typename T>
struct Part {
  const T* head;
  int nhead, nvec, ntail;
  __device__ Part(const T* row, int lo, int hi) {
    head = row + lo;
    const int n = hi - lo;
    const int mis = (int)((16 - (reinterpret_cast<uintptr_t>(head) & 15)) & 15) / (int)sizeof(T);
    nhead = min(n, mis);
    nvec = (n - nhead) / kVec<T>;
    ntail = n - nhead - nvec * kVec<T>;
  }
  __device__ const T* vec(int i) const { return head + nhead + (long long)i * kVec<T>; }
  // single elements are numbered 0 .. nhead + ntail - 1
  __device__ int singles() const { return nhead + ntail; }
  __device__ int single_at(int i) const { return i < nhead ? i : i + nvec * kVec<T>; }  // offset from head
};

// Calls f(x, v) for every element of the part, which begins at index lo.
template <int NT, typename T, typename F>
__device__ __forceinline__ void for_each(const Part<T>& p, int lo, F f) {
  for (int i = threadIdx.x; i < p.nvec; i += NT) {
    float v[kVec<T>];
    unpack(ld_stream(p.vec(i)), v, T{});
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) f(v[k], lo + p.nhead + i * kVec<T> + k);
  }
  if ((int)threadIdx.x < p.singles()) {
    const int o = p.single_at(threadIdx.x);
    f(to_f32(p.head[o]), lo + o);
  }
}

// -------------------------------------------------------------- statistics --
// The careful statistic: any values, one element at a time.
template <int NT, typename T, bool U>
__device__ __noinline__ Stat part_stat_any(const Part<T>& p, float c) {
  Stat t{NEG_INF, 0.f, 0.f};
  for_each<NT>(p, 0, [&](float x, int) {
    if (x > t.m) {
      const float d = fmaxf((t.m - x) * c, kLeast), f = ex2(d);
      t.u = f * (t.u + t.s * d);
      t.s *= f;
      t.m = x;
    }
    const float d = (x - finite_max(t.m)) * c, e = ex2(d);
    t.s += e;
    t.u = fmaf(e, fmaxf(d, kLeast), t.u);  // 0 for a masked logit
  });
  return t;
}

// The fast statistic starts from the maximum kFloor, so that x - m is always
// finite: a logit far below it (a mask) adds 2^-huge = 0.  It does not hold
// for rows without a logit above kFloor, nor for scales that make kFloor
// small or huge, nor its moment for a maximum so far above kFloor that the
// distance passes the range (0 times it is NaN); those take the careful one.
constexpr float kFloor = -9.9499216e29f;  // 0xF1490000: also a bf16
constexpr float kLeastScale = 1e-20f, kMostScale = 1e6f, kMostScaledMax = 1e38f;

struct Run {
  float m;
  float2 s, u;  // two interleaved sums
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// max(a, b) that is NaN where either is, always the same one: a positive NaN,
// which warp_max_f takes as the largest number.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// max(a, kFloor) that keeps a NaN.
__device__ __forceinline__ float floor_nan(float a) { return max_nan(a, kFloor); }

template <typename T, int N>
__device__ __forceinline__ float max_of(const uint4 (&r)[N]) {
  if constexpr (sizeof(T) == 4) {
    float m = kFloor;
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r[i].x), __uint_as_float(r[i].y)),
                         fmaxf(__uint_as_float(r[i].z), __uint_as_float(r[i].w))));
    return m;
  } else {
    uint32_t m = max2(max2(r[0].x, r[0].y, T{}), max2(r[0].z, r[0].w, T{}), T{});
#pragma unroll
    for (int i = 1; i < N; ++i) m = max2(m, max2(max2(r[i].x, r[i].y, T{}), max2(r[i].z, r[i].w, T{}), T{}), T{});
    const float2 f = unpack2(m, T{});
    return fmaxf(f.x, f.y);
  }
}

__device__ __forceinline__ void raise(Run& t, float m, float c, bool u) {
  if (m > t.m) {
    const float d = fmaxf((t.m - m) * c, kLeast), f = ex2(d);
    if (u) {
      t.u.x = f * fmaf(t.s.x, d, t.u.x);
      t.u.y = f * fmaf(t.s.y, d, t.u.y);
    }
    t.s.x *= f;
    t.s.y *= f;
    t.m = m;
  }
}

template <bool U>
__device__ __forceinline__ void add_pair(Run& t, float2 x, float2 neg_m, float2 c2) {
  if (U) {  // 0 * -inf is no term: masked logits are lifted to kFloor
    x.x = floor_nan(x.x);
    x.y = floor_nan(x.y);
  }
  const float2 d = mul2(add2(x, neg_m), c2);
  const float2 e = make_float2(ex2(d.x), ex2(d.y));
  t.s = add2(t.s, e);
  if (U) t.u = fma2(e, d, t.u);
}

// Adds vectors of maximum `most`.
template <typename T, bool U, int N>
__device__ __forceinline__ void add_vectors(Run& t, const uint4 (&r)[N], float most, float c) {
  raise(t, most, c, U);
  const float2 nm = both(-t.m), c2 = both(c);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 4) {
      add_pair<U>(t, make_float2(__uint_as_float(r[i].x), __uint_as_float(r[i].y)), nm, c2);
      add_pair<U>(t, make_float2(__uint_as_float(r[i].z), __uint_as_float(r[i].w)), nm, c2);
    } else {
      add_pair<U>(t, unpack2(r[i].x, T{}), nm, c2);
      add_pair<U>(t, unpack2(r[i].y, T{}), nm, c2);
      add_pair<U>(t, unpack2(r[i].z, T{}), nm, c2);
      add_pair<U>(t, unpack2(r[i].w, T{}), nm, c2);
    }
  }
}

template <typename T, bool U>
__device__ __forceinline__ Stat finish(Run& t, const Part<T>& p, float c) {
  if ((int)threadIdx.x < p.singles()) {
    const float x = to_f32(p.head[p.single_at(threadIdx.x)]);
    raise(t, fmaxf(x, kFloor), c, U);
    const float d = (floor_nan(x) - t.m) * c, e = ex2(d);
    t.s.x += e;
    if (U) t.u.x = fmaf(e, d, t.u.x);
  }
  return Stat{t.m, t.s.x + t.s.y, t.u.x + t.u.y};
}

__device__ __forceinline__ float warp_max_f(float v) {
  // as signed numbers of the same order, in one instruction
  int b = __float_as_int(v);
  b ^= (b >> 31) & 0x7FFFFFFF;
  b = __reduce_max_sync(0xffffffffu, b);
  return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF));
}

// Terms of a part brought to the reference point of a larger set.
__device__ __forceinline__ void rescale(Stat& t, float m, float c) {
  const float d = fmaxf((t.m - finite_max(m)) * c, kLeast), f = ex2(d);
  t.u = f * fmaf(t.s, d, t.u);
  t.s *= f;
  t.m = m;
}

// T^2 sum p (log p - log q), given gap = sum p (teacher - x) relative to their
// maxima and l2 = log2 sum 2^.. of the logits less that of the teacher: each
// part is multiplied by T as often as it has to be and never divided by it.
__device__ __forceinline__ float loss_of(float gap, float l2, float temperature) {
  return temperature * (gap + temperature * (kLn2 * l2));
}

// f of each pair of a vector of logits, rounded to their type.
template <typename T, typename F>
__device__ __forceinline__ uint4 map_vector(uint4 r, F f) {
  if constexpr (sizeof(T) == 4) {
    const float2 a = f(make_float2(__uint_as_float(r.x), __uint_as_float(r.y)));
    const float2 b = f(make_float2(__uint_as_float(r.z), __uint_as_float(r.w)));
    r = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  } else {
    r = make_uint4(pack2_of(f(unpack2(r.x, T{})), T{}), pack2_of(f(unpack2(r.y, T{})), T{}),
                   pack2_of(f(unpack2(r.z, T{})), T{}), pack2_of(f(unpack2(r.w, T{})), T{}));
  }
  return r;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Logits of a block's part when C blocks share a row: whole multiples of 64,
// so that aligned rows have aligned parts.
__host__ __device__ __forceinline__ int part_len(int V, int C) { return (((V + C - 1) / C) + 63) & ~63; }

// Starts [from, to), or its first `most` bytes, on its way to L2 (one thread).
__device__ __forceinline__ void prefetch_bytes(const void* from, const void* to, int most) {
  if (threadIdx.x != 0) return;
  const uintptr_t p = (reinterpret_cast<uintptr_t>(from) + 15) & ~(uintptr_t)15, e = reinterpret_cast<uintptr_t>(to);
  if (p + 16 > e) return;
  const uint32_t bytes = (uint32_t)min((unsigned long long)most, (unsigned long long)(e - p)) & ~15u;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// The same for the next part that a block of this place will take, while this
// one has no more loads to make: blocks that began together are in their
// joins and selections together, and HBM would idle meanwhile.
template <typename T>
__device__ __forceinline__ void prefetch_part(const RowArgs& a, long long row, int lo, int hi, int most) {
  const long long next = row + a.ahead;
  if (a.ahead == 0 || next >= a.rows || lo >= hi) return;
  const T* x = static_cast<const T*>(a.x) + next * a.x_stride;
  prefetch_bytes(x + lo, x + hi, most);
}

}  // namespace
}  // namespace ibwd
