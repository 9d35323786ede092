// Operators over rows of logits on sm_103a: log probabilities, entropy and
// top alternatives, their gradient, and the distillation loss from a
// teacher's top logits with its gradient.
//
// A row x of V logits has, with c = log2(e) / temperature,
//   m = max x,  d_v = (x_v - m) c,  s = sum 2^d_v,  u = sum 2^d_v d_v
//   lse = m / temperature + ln 2 log2 s,  log2 p_v = d_v - log2 s,
//   entropy = ln 2 (log2 s - u / s)
// and every function of the row follows from (m, s, u) and single logits.
// (m, s, u) of disjoint parts join exactly like running ones: both are scaled
// to the larger maximum.
//
// A cluster of C thread blocks takes a row, each block a contiguous part; the
// parts' statistics are exchanged through distributed shared memory and
// joined in the blocks' order, so few rows still fill the machine and every
// result is bitwise reproducible.
//
// Bound by HBM when an element costs few enough instructions: unpacking, the
// maximum, two packed operations for d, one exponential and one or two packed
// sums.
#include <cooperative_groups.h>

#include <algorithm>

#include "logits.cuh"

namespace cg = cooperative_groups;

namespace ibwd {
namespace {

constexpr int kMaxThreads = 256;  // of a block: 256 for long rows, 128 or 64 for short ones
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxTop = 128;
template <int NT>
constexpr int kBlocks = 1024 / NT;  // of an SM
// Bytes of the next row that come to L2 early (2048 rows of 131072 bf16, 64
// alternatives: 99.6 us with 16 KB, 98.8 with 32, 101.9 with 64; none: 128).
constexpr int kAhead = 32 * 1024;
constexpr int kSmallPart = 32 * 1024, kTinyPart = 8 * 1024;
constexpr int kCand = 1024;    // candidates a block ranks for the top alternatives
constexpr int kSegments = 16;  // maxima a thread keeps of its logits

// Order of the logits as unsigned numbers (-0 counts as +0).
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Maxima of a thread's vectors in runs of 1 << bits of them, at most
// kSegments, by the upper half of their order: single vectors of short rows,
// else multiples of kUnroll.
template <int NT>
struct Segments {
  uint16_t* at;  // [kSegments][NT], or nullptr
  int bits;
  float run;
  template <typename T>
  __device__ Segments(uint16_t* a, const Part<T>& p) : at(a), bits(0), run(NEG_INF) {
    static_assert(kUnroll == 4, "two bits");
    const int vectors = (p.nvec + NT - 1) / NT;  // of a thread
    if (vectors > kSegments) bits = 2;
    while ((vectors - 1) >> bits >= kSegments) ++bits;
  }
  __device__ __forceinline__ bool single() const { return bits == 0; }
  // vector number `v` of the thread; a run begins where v is a multiple of its
  // length, from kFloor (the bits of a NaN, where a run holds nothing else, are
  // no maximum)
  __device__ __forceinline__ void put(int v, float most) {
    run = fmaxf((v & ((1 << bits) - 1)) ? run : kFloor, most);
    at[(v >> bits) * NT + threadIdx.x] = (uint16_t)(order_bits(run) >> 16);
  }
};

// Streamed from global memory, the next vectors' loads ahead of the sums.
template <int NT, typename T, bool U, bool TOP>
__device__ __forceinline__ Stat part_stat(const Part<T>& p, Segments<NT>& seg, float c) {
  Run t{kFloor, {0.f, 0.f}, {0.f, 0.f}};
  int i = threadIdx.x, v = 0;  // the thread's next vector, and its number
  constexpr int kStep = kUnroll * NT;
  auto four = [&](const uint4(&r)[kUnroll]) {
    const float most = max_of<T>(r);
    if (TOP) {
      if (seg.single()) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const uint4 one[1] = {r[k]};
          seg.put(v + k, max_of<T>(one));
        }
      } else {
        seg.put(v, most);
      }
      v += kUnroll;
    }
    add_vectors<T, U>(t, r, most, c);
  };
  if (i + (kUnroll - 1) * NT < p.nvec) {
    uint4 r[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) r[k] = ld_stream(p.vec(i + k * NT));
    for (i += kStep; i + (kUnroll - 1) * NT < p.nvec; i += kStep) {
      uint4 n[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) n[k] = ld_stream(p.vec(i + k * NT));
      four(r);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) r[k] = n[k];
    }
    four(r);
  }
  if (i < p.nvec) {
    float all = NEG_INF;
    int first = v;
    for (; i < p.nvec; i += NT) {
      const uint4 r[1] = {ld_stream(p.vec(i))};
      const float most = max_of<T>(r);
      all = fmaxf(all, most);
      if (TOP && seg.single()) seg.put(v++, most);
      add_vectors<T, U>(t, r, most, c);
    }
    if (TOP && !seg.single()) seg.put(first, all);
  }
  return finish<T, U>(t, p, c);
}

struct Stage {
  float m[kMaxWarps], s[kMaxWarps], u[kMaxWarps];
  Stat of_block[kMaxCluster];
};

// The statistic of the row in every thread of its blocks: the maximum first,
// then sums in the order of lanes, warps and blocks.  most: the maximum of
// this block's part.
template <int NT, bool U>
__device__ __forceinline__ Stat row_stat(Stat t, float c, Stage& st, int C, float& most) {
  constexpr int NW = NT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float wm = warp_max_f(t.m);
  __syncthreads();
  if (lane == 0) st.m[warp] = wm;
  __syncthreads();
  float m = st.m[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) m = fmaxf(m, st.m[w]);
  most = m;
  rescale(t, m, c);
  t.s = warp_sum(t.s);
  if (U) t.u = warp_sum(t.u);
  if (lane == 0) {
    st.s[warp] = t.s;
    if (U) st.u[warp] = t.u;
  }
  __syncthreads();
  t.s = t.u = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    t.s += st.s[w];
    if (U) t.u += st.u[w];
  }
  if (C == 1) return t;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();  // every block has started, and is done with an earlier exchange
  if ((int)threadIdx.x < C) *cl.map_shared_rank(&st.of_block[cl.block_rank()], threadIdx.x) = t;
  cl.sync();
  m = st.of_block[0].m;
  for (int i = 1; i < C; ++i) m = fmaxf(m, st.of_block[i].m);
  Stat r{m, 0.f, 0.f};
  for (int i = 0; i < C; ++i) {
    Stat o = st.of_block[i];
    rescale(o, m, c);
    r.s += o.s;
    r.u += o.u;
  }
  return r;
}

// ------------------------------------------------------- top alternatives --
// Candidates as one unsigned key: larger logit first, then lower index.
__device__ __forceinline__ unsigned long long order_key(float x, int v) {
  return ((unsigned long long)order_bits(x) << 32) | (uint32_t)~v;
}

constexpr int kHot = 1024;       // segments looked at again
constexpr int kDistances = 256;  // distances of the maxima from the largest that are counted

template <int NT>
struct TopShared {
  alignas(16) unsigned long long cand[kCand + 4];
  unsigned long long merge[kMaxTop * kMaxCluster];
  int merge_n[kMaxCluster];
  uint16_t segment[kSegments * NT];
  int count_at[kDistances];  // maxima by their distance from the largest one
  int hot[kHot];
  int nhot, ncand;
  uint32_t least, below;
  uint32_t bound;  // upper half of an order
  int warp_n[kMaxWarps];
};

// The rare case of more than kCand entries at or above the bound (many equal
// logits, or logits whose order follows the threads): the exact order of the
// n-th largest by bisection, then everything above it and the equal ones of
// lowest index.
template <int NT, typename T>
__device__ __noinline__ void top_exact(const Part<T>& p, int lo, int hi, int n, uint32_t bound, TopShared<NT>& sh) {
  // masked logits and NaN are no entries
  auto order = [](float x) { return x > NEG_INF ? order_bits(x) : 0u; };
  // entries of the part above `cut`: their number, the least of them, and the
  // largest at or below it
  auto above = [&](uint32_t cut, uint32_t& least, uint32_t& below) {
    __syncthreads();
    if (threadIdx.x == 0) {
      sh.ncand = 0;
      sh.least = ~0u;
      sh.below = 0;
    }
    __syncthreads();
    int k = 0;
    uint32_t l = ~0u, h = 0;
    for_each<NT>(p, lo, [&](float x, int) {
      const uint32_t key = order(x);
      if (key > cut) {
        ++k;
        l = min(l, key);
      } else {
        h = max(h, key);
      }
    });
    if (k) atomicAdd(&sh.ncand, k);
    atomicMin(&sh.least, l);
    atomicMax(&sh.below, h);
    __syncthreads();
    least = sh.least;
    below = sh.below;
    return sh.ncand;
  };
  // entries above a: `count`, at least n of them while over kCand; entries
  // above b: fewer than n.  Both move to the nearest entries that occur.
  uint32_t a = bound, b = ~0u, least, below;
  int count = above(a, least, below);
  bool equal = false;  // a is the n-th largest itself
  while (count > kCand) {
    a = least - 1;
    if (b - a == 1) {  // more than kCand entries are equal to b
      a = b;
      equal = true;
      break;
    }
    const uint32_t mid = a + (b - a) / 2;
    uint32_t l;
    const int k = above(mid, l, below);
    if (k >= n) {
      a = mid;
      count = k;
      least = l;
    } else {
      b = below;  // (some entry lies in (a, mid])
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.ncand = 0;
  __syncthreads();
  for_each<NT>(p, lo, [&](float x, int v) {
    if (order(x) > a) sh.cand[atomicAdd(&sh.ncand, 1)] = order_key(x, v);
  });
  __syncthreads();
  if (!equal) return;
  // the lowest indices among the equal ones, in order
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int have = sh.ncand;
  for (int v0 = lo; v0 < hi && have < n; v0 += NT) {
    const int v = v0 + threadIdx.x;
    const bool eq = v < hi && order(to_f32(p.head[v - lo])) == a;
    const unsigned mask = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) sh.warp_n[warp] = __popc(mask);
    __syncthreads();
    int at = have + __popc(mask & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) at += sh.warp_n[w];
      total += sh.warp_n[w];
    }
    if (eq && at < n) sh.cand[at] = ((unsigned long long)a << 32) | (uint32_t)~v;
    have += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) sh.ncand = min(have, n);
  __syncthreads();
}

// The n largest entries of this block's part, as sorted keys in
// out[0 .. return value), from the threads' own maxima: the n-th largest of
// those bounds the n-th largest entry from below (they are maxima of disjoint
// sets), and only segments whose maximum reaches the bound can hold an entry
// that does, so the second look reads a few of them (a 131072-logit row: some
// 80 of 4096).  The bound is found to the upper 16 bits of its order (all of
// a bf16) by counting the maxima at each distance from the largest, or by
// bisection where it is further away than that.
// sh.count_at is zero and sh.nhot, sh.ncand are 0 on entry.
template <int NT, typename T>
__device__ __forceinline__ int part_top(const Part<T>& p, int lo, int hi, int n, float my_max, float most, int bits,
                                        TopShared<NT>& sh, unsigned long long* out) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t my_key = order_bits(my_max) >> 16, top_key = order_bits(most) >> 16;
  const int mine = p.nvec > t ? (p.nvec - t + NT - 1) / NT : 0;  // vectors of this thread
  const int segments = (mine + (1 << bits) - 1) >> bits;
  // Short rows count their vectors' maxima where the threads' own are too few
  // to bound n entries well; a thread's single elements are left out of those.
  // (2432 rows of 32768 bf16 in 256 threads, 8 alternatives: 47 us by the
  // vectors' maxima, 43 by the threads'; 128 alternatives: 57 and 60.)
  const bool fine = bits == 0 && 2 * n >= NT;
  if (fine) {
    for (int s = 0; s < segments; ++s) {
      const uint32_t d = top_key - sh.segment[s * NT + t];
      if (d < kDistances) atomicAdd(&sh.count_at[d], 1);
    }
  } else if (top_key - my_key < kDistances) {
    atomicAdd(&sh.count_at[top_key - my_key], 1);
  }
  __syncthreads();
  if (t < 32) {
    // lane i has distances 8 i .. 8 i + 7
    constexpr int PER = kDistances / 32;
    int c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = sh.count_at[lane * PER + i];
      sum += c[i];
    }
    int upto = sum;  // maxima at the distances of this lane and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned reach = __ballot_sync(0xffffffffu, upto >= n);
    if (reach == 0) {
      if (lane == 0) sh.bound = ~0u;
    } else if (lane == __ffs(reach) - 1) {
      int have = upto - sum, d = lane * PER;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (have < n) {
          have += c[i];
          d = lane * PER + i;
        }
      sh.bound = top_key - d;
    }
  }
  __syncthreads();
  if (sh.bound == ~0u) {  // uniform: bisection over all 16 bits
    uint32_t key = 0;
    for (uint32_t bit = 1u << 15; bit; bit >>= 1) {
      unsigned k = my_key >= (key | bit);
      if (fine) {
        k = 0;
        for (int s = 0; s < segments; ++s) k += sh.segment[s * NT + t] >= (key | bit);
      }
      if (t == 0) sh.least = 0;
      __syncthreads();
      k = __reduce_add_sync(0xffffffffu, k);
      if (lane == 0 && k) atomicAdd(&sh.least, k);
      __syncthreads();
      if (sh.least >= (unsigned)n) key |= bit;
      __syncthreads();
    }
    if (t == 0) sh.bound = key;
    __syncthreads();
  }
  // (a thread without logits above kFloor stops there: no bound then)
  const uint32_t half = sh.bound > order_bits(kFloor) >> 16 ? sh.bound : 0;
  const uint32_t bound = max(half << 16, order_bits(NEG_INF) + 1);
  const float cut = half ? order_value(bound) : NEG_INF;
  auto wanted = [&](float x) { return half ? x >= cut : x > cut; };
  // Places for the set bits of every lane's mask behind `count`: one addition
  // a warp; put(place, bit) for each.
  auto append = [&](int& count, unsigned mask, auto put) {
    const int mine = __popc(mask);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    int base = 0;
    if (lane == 31 && upto) base = atomicAdd(&count, upto);
    base = __shfl_sync(0xffffffffu, base, 31) + upto - mine;
    for (; mask; mask &= mask - 1, ++base) put(base, __ffs(mask) - 1);
  };
  {
    unsigned mask = 0;
    if (my_key >= half) {
#pragma unroll
      for (int s = 0; s < kSegments; ++s)
        mask |= s < segments && sh.segment[s * NT + t] >= half ? 1u << s : 0u;
    }
    append(sh.nhot, mask, [&](int at, int s) {
      if (at < kHot) sh.hot[at] = s * NT + t;
    });
  }
  __syncthreads();
  const int nhot = sh.nhot;
  if (nhot <= kHot) {
    const int items = nhot << bits;
    constexpr int V = kVec<T>, TAKE = kUnroll;  // vectors a lane takes together: 32 values at most
    for (int e0 = warp * 32; e0 < items; e0 += TAKE * NT) {
      uint4 r[TAKE];
      int at[TAKE];
#pragma unroll
      for (int k = 0; k < TAKE; ++k) {
        const int e = e0 + lane + k * NT;
        at[k] = p.nvec;
        if (e < items) {
          const int h = sh.hot[e >> bits];
          at[k] = h % NT + (((h / NT) << bits) + (e & ((1 << bits) - 1))) * NT;
        }
        if (at[k] < p.nvec) r[k] = ld_stream(p.vec(at[k]));
      }
      unsigned mask = 0;
#pragma unroll
      for (int k = 0; k < TAKE; ++k)
        if (at[k] < p.nvec) {
          float v[V];
          unpack(r[k], v, T{});
#pragma unroll
          for (int j = 0; j < V; ++j) mask |= wanted(v[j]) ? 1u << (k * V + j) : 0u;
        }
      append(sh.ncand, mask, [&](int place, int i) {
        // element i % V of vector i / V
        uint4 q = r[0];
        int vec = at[0];
#pragma unroll
        for (int k = 1; k < TAKE; ++k)
          if (i / V == k) {
            q = r[k];
            vec = at[k];
          }
        const int word = i % V * (int)sizeof(T) / 4;
        const uint32_t w = word == 0 ? q.x : word == 1 ? q.y : word == 2 ? q.z : q.w;
        float x;
        if constexpr (sizeof(T) == 4)
          x = __uint_as_float(w);
        else
          x = i & 1 ? unpack2(w, T{}).y : unpack2(w, T{}).x;
        if (place < kCand) sh.cand[place] = order_key(x, lo + p.nhead + vec * V + i % V);
      });
    }
    if (warp == 0) {
      const int o = lane < p.singles() ? p.single_at(lane) : 0;
      const float x = lane < p.singles() ? to_f32(p.head[o]) : NEG_INF;
      append(sh.ncand, wanted(x) ? 1u : 0u, [&](int place, int) {
        if (place < kCand) sh.cand[place] = order_key(x, lo + o);
      });
    }
  }
  __syncthreads();
  if (nhot > kHot || sh.ncand > kCand) top_exact<NT>(p, lo, hi, n, bound - 1, sh);  // uniform
  const int count = sh.ncand;
  if (t < 4) sh.cand[count + t] = 0;  // below every key: they are read four at a time, by two lanes
  __syncthreads();
  for (int i0 = 0; i0 < count; i0 += NT / 2) {
    const int i = i0 + (t >> 1);
    if (i0 + (warp << 4) >= count) break;  // uniform in a warp
    const unsigned long long key = i < count ? sh.cand[i] : ~0ull;
    int r = 0;
#pragma unroll 4
    for (int k = 2 * (t & 1); k < count; k += 4) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sh.cand[k]);
      r += (o.x > key) + (o.y > key);
    }
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    if (i < count && !(t & 1) && r < n) out[r] = key;
  }
  return min(count, n);
}

// --------------------------------------------------------------- gradients --
// Writes the gradient of this block's part, f of each pair of logits: by
// vectors where logits and gradient lie alike in their 16-byte blocks.
// dst: the gradient of p.head[0].
template <int NT, typename T, typename F>
__device__ __forceinline__ void map_part(const Part<T>& p, T* dst, F f) {
  const bool alike = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(p.head)) & 15) == 0;
  if (alike) {
    T* dv = dst + p.nhead;
    auto give = [&](int i, uint4 r) {
      st_stream(dv + (long long)i * kVec<T>, map_vector<T>(r, f));
    };
    int i = threadIdx.x;
    for (; i + (kUnroll - 1) * NT < p.nvec; i += kUnroll * NT) {
      uint4 r[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) r[k] = ld_stream(p.vec(i + k * NT));
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) give(i + k * NT, r[k]);
    }
    for (; i < p.nvec; i += NT) give(i, ld_stream(p.vec(i)));
    if ((int)threadIdx.x < p.singles()) {
      const int o = p.single_at(threadIdx.x);
      dst[o] = from_f32<T>(f(both(to_f32(p.head[o]))).x);
    }
  } else {
    const int n = p.singles() + p.nvec * kVec<T>;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += NT) dst[i] = from_f32<T>(f(both(to_f32(p.head[i]))).x);
  }
}

struct Kept {  // [K] each, in shared memory
  int* id;   // kept token, or -1
  float* p;  // the teacher's value, then kShare 2^((value - max) c)
  float* x;  // the student's logit of it (read by the thread that wrote it)
};

template <typename T, RowOp OP, bool TOP, int NT>
__global__ void __launch_bounds__(NT, kBlocks<NT>) rows_kernel(RowArgs a, int C) {
  constexpr int NW = NT / 32;
  constexpr bool kDistill = OP == RowOp::kDistillFwd || OP == RowOp::kDistillBwd || OP == RowOp::kDistillGrad;
  constexpr bool kStat = OP == RowOp::kLogpFwd || OP == RowOp::kDistillFwd || OP == RowOp::kDistillGrad;
  constexpr bool kEntropy = OP == RowOp::kLogpFwd;
  __shared__ Stage stage;
  __shared__ float kept_max[kMaxWarps], kept_z[kMaxWarps], kept_gap[kMaxWarps];
  extern __shared__ __align__(16) unsigned char raw[];  // TopShared, or the kept tokens
  TopShared<NT>& top = *reinterpret_cast<TopShared<NT>*>(raw);
  Kept kept;
  kept.id = reinterpret_cast<int*>(raw);
  kept.p = reinterpret_cast<float*>(kept.id + a.K);
  kept.x = kept.p + a.K;

  const int rank = C == 1 ? 0 : (int)(blockIdx.x % C);
  const long long row = blockIdx.x / C;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int len = part_len(a.V, C);
  const int lo = (int)min((long long)a.V, (long long)rank * len), hi = (int)min((long long)a.V, (long long)lo + len);
  const T* xr = static_cast<const T*>(a.x) + row * a.x_stride;
  const Part<T> part(xr, lo, hi);
  const float inv_t = 1.f / a.temperature, c = kLog2e / a.temperature;

  // (a gradient's logits come to L2 while its first small loads arrive)
  if (!kStat) prefetch_bytes(xr + lo, xr + hi, kAhead);
  // what the row needs besides its logits is on its way before them
  int token = -1;
  if (OP == RowOp::kLogpFwd && rank == 0 && t == 0 && a.tokens) token = a.tokens[row];
  if (kDistill) {
    for (int j = t; j < a.K; j += NT) {
      cp_async4(smem_u32(kept.id + j), a.ids + row * a.K + j);
      cp_async4(smem_u32(kept.p + j), a.teacher + row * a.K + j);
    }
    cp_async_commit();
  }

  Stat st{0.f, 1.f, 0.f};
  float my_max = NEG_INF, most = NEG_INF;  // of the thread's and of the block's logits
  Segments<NT> segments(TOP ? top.segment : nullptr, part);
  Stat own{NEG_INF, 0.f, 0.f};
  if (kStat) {
    own = part_stat<NT, T, kEntropy, TOP>(part, segments, c);
    my_max = own.m;
  }
  if (kStat) prefetch_part<T>(a, row, lo, hi, kAhead);
  // The student's logits of the teacher's slots (without the loss, of those
  // in this part); the first one of a thread is used after the row's statistic
  // and comes in meanwhile.
  float x_first = 0.f;
  if (kDistill) {
    cp_async_wait_all();
    float tmax = NEG_INF;
    for (int j = t; j < a.K; j += NT) {
      const int id = kept.id[j];
      const bool ok = id >= 0 && id < a.V;
      const bool used = OP == RowOp::kDistillBwd ? id >= lo && id < hi : ok;
      const float x = used ? to_f32(xr[id]) : 0.f;
      if (ok)
        tmax = max_nan(tmax, kept.p[j]);
      else {
        kept.id[j] = -1;
        kept.p[j] = NEG_INF;
      }
      if (j == t)
        x_first = x;
      else
        kept.x[j] = x;
    }
    tmax = warp_max_f(tmax);
    if (lane == 0) kept_max[warp] = tmax;
    if (!kStat) __syncthreads();  // (the statistic has barriers of its own)
  }
  float x_token = 0.f;
  if (OP == RowOp::kLogpFwd && token >= 0 && token < a.V) x_token = to_f32(xr[token]);
  if (kStat) {
    if (TOP) {  // (before the statistic's barriers)
      for (int i = t; i < kDistances; i += NT) top.count_at[i] = 0;
      if (t == 0) top.nhot = top.ncand = 0;
    }
    st = row_stat<NT, kEntropy>(own, c, stage, C, most);
    if (!(st.m > kFloor) || c < kLeastScale || c > kMostScale || (kEntropy && st.m * c > kMostScaledMax)) {
      // (uniform over the cluster)
      float ignored;
      st = row_stat<NT, kEntropy>(part_stat_any<NT, T, kEntropy>(part, c), c, stage, C, ignored);
    }
  }
  // log2 p_v = (x_v - ref) c - l2s
  float ref, l2s;
  bool empty;  // every logit masked
  if (kStat) {
    empty = st.m == NEG_INF && st.s == 0.f;  // (s is NaN when the row holds a NaN)
    ref = finite_max(st.m);
    l2s = log2f(st.s);
  } else {
    // x / T - lse as (x - lse T) / T, lse T in two parts: the difference is
    // rounded, not its terms, which for a row of the type's lowest value pass
    // the range, and at T = 1e-3 are some 1e4
    const float lse = a.lse[row];
    empty = lse == NEG_INF;
    ref = lse * a.temperature;
    l2s = c * fmaf(lse, a.temperature, -ref);
    if (isinf(ref)) {
      if (!isinf(lse)) ref = copysignf(kLargest, ref);
      l2s = 0.f;
    }
  }

  if (OP == RowOp::kLogpFwd) {
    if (rank == 0 && t == 0) {
      if (a.lse) a.lse[row] = empty ? NEG_INF : ref * inv_t + kLn2 * l2s;
      if (a.entropy) a.entropy[row] = empty ? 0.f : kLn2 * (l2s - st.u / st.s);
      if (a.tokens) {
        float lp = 0.f;
        if (token >= 0 && token < a.V) lp = empty ? NEG_INF : (x_token - ref) * inv_t - kLn2 * l2s;
        a.logprob[row] = lp;
      }
    }
    if (TOP) {
      const int n = a.top_n;
      auto put = [&](int i, unsigned long long key) {
        a.top_ids[row * n + i] = (int)~(uint32_t)key;
        a.top_logprobs[row * n + i] = (order_value((uint32_t)(key >> 32)) - ref) * inv_t - kLn2 * l2s;
      };
      int total = 0;
      if (C == 1) {
        total = part_top<NT>(part, lo, hi, n, my_max, most, segments.bits, top, top.merge);
        __syncthreads();
        for (int i = t; i < total; i += NT) put(i, top.merge[i]);
      } else {
        cg::cluster_group cl = cg::this_cluster();
        const int count = part_top<NT>(part, lo, hi, n, my_max, most, segments.bits, top,
                                   cl.map_shared_rank(top.merge, 0) + rank * kMaxTop);
        if (t == 0) *(cl.map_shared_rank(top.merge_n, 0) + rank) = count;
        cl.sync();
        if (rank != 0) return;
        for (int i = 0; i < C; ++i) total += top.merge_n[i];
        // place of an entry: its own place plus, in every other sorted list,
        // the number of larger keys
        for (int e = t; e < C * n; e += NT) {
          const int l = e / n, i = e % n;
          if (i >= top.merge_n[l]) continue;
          const unsigned long long key = top.merge[l * kMaxTop + i];
          int r = i;
          for (int k = 0; k < C; ++k) {
            if (k == l) continue;
            int x0 = 0, x1 = top.merge_n[k];
            while (x0 < x1) {
              const int mid = (x0 + x1) >> 1;
              if (top.merge[k * kMaxTop + mid] > key)
                x0 = mid + 1;
              else
                x1 = mid;
            }
            r += x0;
          }
          if (r < n) put(r, key);
        }
      }
      for (int i = total + t; i < n; i += NT) {
        a.top_ids[row * n + i] = -1;
        a.top_logprobs[row * n + i] = isnan(l2s) ? l2s : NEG_INF;
      }
    }
    return;
  }

  T* dst = static_cast<T*>(a.dx) + row * a.dx_stride + lo;
  if (OP == RowOp::kLogpBwd) {
    const int id = a.tokens ? a.tokens[row] : -1;
    const bool tok = id >= 0 && id < a.V && a.dlogprob != nullptr;
    const float g = tok ? a.dlogprob[row] * inv_t : 0.f;
    const float b = a.dentropy ? a.dentropy[row] * inv_t : 0.f;
    const float h = a.dentropy ? a.entropy[row] : 0.f;
    const bool here = tok && id >= lo && id < hi;
    const float xt = here ? to_f32(xr[id]) : 0.f;
    __syncthreads();  // the logit is read before its place may be overwritten
    if (empty) {
      map_part<NT>(part, dst, [](float2) { return both(0.f); });
      return;
    }
    // -p (g + b (log p + h)), log2 p = d - l2s: the part l2s is in the factors
    const float f = ex2(-l2s), b2 = -b * kLn2;
    const float2 c2 = both(c), nref = both(-ref), k0 = both(f * -fmaf(b2, l2s, fmaf(b, h, g))), k1 = both(f * b2);
    auto grad = [&](float2 x) {
      float2 d = mul2(add2(x, nref), c2);
      const float2 p = make_float2(ex2(d.x), ex2(d.y));
      d.x = fmaxf(d.x, kLeast);
      d.y = fmaxf(d.y, kLeast);
      return mul2(p, fma2(d, k1, k0));
    };
    map_part<NT>(part, dst, grad);
    __syncthreads();
    if (t == 0 && here) dst[id - lo] = from_f32<T>(g + grad(both(xt)).x);
    return;
  }

  if (kDistill) {
    // p_j = w_j / z with w_j = kShare 2^((teacher_j - tmax) c)
    float tmax = kept_max[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) tmax = max_nan(tmax, kept_max[w]);
    const bool zero = tmax == NEG_INF || empty;
    const float tref = finite_max(tmax);
    float z = 0.f, gap = 0.f;
    if (warp * 32 < a.K) {
      for (int j = t; j < a.K; j += NT) {
        const float d = kept.p[j] - tref;
        const float w = ex2(d * c) * kShare;
        z += w;
        // in the logits' units: a lowest-value mask stays finite there
        const float x = j == t ? x_first : kept.x[j];
        if (w > 0.f) gap += w * (d - (x - ref));
        kept.p[j] = w;
      }
      z = warp_sum(z);
      gap = warp_sum(gap);
    }
    if (lane == 0) {
      kept_z[warp] = z;
      kept_gap[warp] = gap;
    }
    if (OP != RowOp::kDistillFwd) {
      // (every logit of a kept token has been read, by this block or, with
      // statistics, before the blocks met)
      float g = a.dloss ? a.dloss[row] * a.temperature : a.temperature;
      if (OP == RowOp::kDistillGrad) g *= a.grad_scale;
      const float2 c2 = both(c), nref = both(-ref), off = both(-l2s), g2 = both(g);
      auto grad = [&](float2 x) {
        const float2 d = fma2(add2(x, nref), c2, off);
        return mul2(make_float2(ex2(d.x), ex2(d.y)), g2);
      };
      if (zero)
        map_part<NT>(part, dst, [](float2) { return both(0.f); });
      else
        map_part<NT>(part, dst, grad);
      __syncthreads();
      z = gap = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) z += kept_z[w];
      const float iz = 1.f / z;
      if (!zero)
        for (int j = t; j < a.K; j += NT) {
          const int id = kept.id[j];
          if (id < lo || id >= hi) continue;
          float p = 0.f;
          bool first = true;
#pragma unroll 4
          for (int k = 0; k < a.K; ++k)
            if (kept.id[k] == id) {
              if (k < j) first = false;
              p += kept.p[k];
            }
          if (first) dst[id - lo] = from_f32<T>(grad(both(j == t ? x_first : kept.x[j])).x - g * p * iz);
        }
    } else {
      __syncthreads();
    }
    if (OP != RowOp::kDistillBwd && rank == 0 && t == 0) {
      z = gap = 0.f;
      for (int w = 0; w < NW; ++w) {
        z += kept_z[w];
        gap += kept_gap[w];
      }
      if (a.loss) a.loss[row] = zero ? 0.f : loss_of(gap / z, l2s - log2f(z / kShare), a.temperature);
      if (OP == RowOp::kDistillFwd) a.lse[row] = empty ? NEG_INF : ref * inv_t + kLn2 * l2s;
    }
  }
}

template <typename T, RowOp OP, bool TOP, int NT>
cudaError_t launch_threads(RowArgs a, int C, cudaStream_t st) {
  const size_t smem = TOP ? sizeof(TopShared<NT>) : (size_t)a.K * 12;
  cudaLaunchConfig_t cfg{};
  a.ahead = std::max(1, kBlocks<NT> * a.num_sms / C);
  cfg.gridDim = dim3((unsigned)(a.rows * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  // (the blocks of a row meet for its statistic; without one they only share it)
  cfg.numAttrs = C > 1 && OP != RowOp::kLogpBwd && OP != RowOp::kDistillBwd ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, rows_kernel<T, OP, TOP, NT>, a, C);
}

// Threads of a block by the bytes of its part: a short part costs the latency
// of its steps, and more blocks of fewer threads overlap them (4864 rows of
// 2048 bf16, 64 alternatives: 56 us by 256 threads, 32 by 64) -- unless the
// rows are too few to fill the SMs (8 of 65536: 12.6 us by 128, 9.4 by 256).
// Log probabilities take 128 threads for up to 64 KB (2432 rows of 32768 bf16:
// 28.2 us by 256, 26.8 by 128; 8 alternatives: 43 and 37), but not with many
// alternatives, which as few maxima bound badly (64: 47 and 55); nor do the
// gradients (2048 rows of 65536 in parts of 32768: 81.5 and 82.9).
template <typename T, RowOp OP, bool TOP>
cudaError_t launch_rows_t(const RowArgs& a, int C, cudaStream_t st) {
  const int bytes = part_len(a.V, C) * (int)sizeof(T);
  if (a.rows * C <= 2 * a.num_sms) return launch_threads<T, OP, TOP, 256>(a, C, st);
  if (bytes <= kTinyPart) return launch_threads<T, OP, TOP, 64>(a, C, st);
  const bool more = OP == RowOp::kLogpFwd && (!TOP || a.top_n <= 32);
  if (bytes <= (more ? 2 : 1) * kSmallPart) return launch_threads<T, OP, TOP, 128>(a, C, st);
  return launch_threads<T, OP, TOP, 256>(a, C, st);
}

template <typename T>
cudaError_t launch_typed(RowOp op, const RowArgs& a, cudaStream_t st) {
  // Blocks a row.  Rows that meet in a cluster or select a top pay for each
  // block, so they share only where SMs would be idle, and parts keep some
  // work: 16 KB, or 128 KB with a selection and its merge (4 rows of 131072
  // bf16: 7.4 us in one block each, 4.2 in eight; with 20 alternatives 8 rows
  // of 65536 take 8.2 us in one, 9.7 in two, and one fp32 row of 131072 12.7
  // in one, 9.3 in four, 10.1 in eight).
  // A backward pass has no joins: its blocks take 32 KB at least, and so many
  // that the last ones do not leave the SMs idle for long (4096 rows of 131072
  // bf16: 339 us in one block a row, 315 in two) -- with a teacher's slots,
  // which every block of a row goes through, as many as fill the SMs.
  const bool bwd = op == RowOp::kLogpBwd || op == RowOp::kDistillBwd;
  const bool top = op == RowOp::kLogpFwd && a.top_n;
  const long long blocks = op == RowOp::kLogpBwd      ? 32LL * a.num_sms
                           : op == RowOp::kDistillBwd ? 4LL * a.num_sms
                                                      : a.num_sms;
  const int least = (bwd ? 8 : top ? 32 : 4) * kMaxThreads * kVec<T>;
  int C = 1;
  while (C < kMaxCluster && a.rows * 2 * C <= blocks && a.V >= 2LL * C * least) C *= 2;
  switch (op) {
    case RowOp::kLogpFwd:
      return a.top_n ? launch_rows_t<T, RowOp::kLogpFwd, true>(a, C, st)
                     : launch_rows_t<T, RowOp::kLogpFwd, false>(a, C, st);
    case RowOp::kLogpBwd: return launch_rows_t<T, RowOp::kLogpBwd, false>(a, C, st);
    case RowOp::kDistillFwd: return launch_rows_t<T, RowOp::kDistillFwd, false>(a, C, st);
    case RowOp::kDistillBwd: return launch_rows_t<T, RowOp::kDistillBwd, false>(a, C, st);
    default: return launch_rows_t<T, RowOp::kDistillGrad, false>(a, C, st);
  }
}

}  // namespace

cudaError_t launch_rows(RowOp op, const RowArgs& a, cudaStream_t st) {
  if (!a.rows) return cudaSuccess;
  if (op == RowOp::kDistillGrad && distill_resident(a)) return launch_distill_resident(a, st);
  switch (a.type) {
    case 0: return launch_typed<float>(op, a, st);
    case 1: return launch_typed<__nv_bfloat16>(op, a, st);
    default: return launch_typed<__half>(op, a, st);
  }
}

}  // namespace ibwd
