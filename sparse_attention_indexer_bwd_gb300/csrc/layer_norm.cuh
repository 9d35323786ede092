// Layer norm over the rows of a matrix, forward and backward, on sm_103a:
//   y = (x - mean) rstd gamma + beta,
//   dx = rstd (d - sum(d)/N - xh sum(d xh)/N),  xh = (x - mean) rstd, d = dy gamma,
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy.
// About ten operations an element beside four to twelve bytes: bound by HBM,
// or by the launch where rows are few.
//
// A team of threads holds a row in registers (16 elements a thread at most)
// or, where registers would leave an SM too few threads, in shared memory, so
// every element is read once: 8 to 32 lanes of a warp for short rows, a thread
// block for longer ones.  Teams stay resident and walk the rows; each thread
// copies its own elements of the next rows into its own slots of a
// shared-memory ring (cp.async), so several rows are in flight without
// registers or barriers.  The weights stay in registers or shared memory, the
// backward pass's column sums of the team's rows in registers.  Those meet in
// a fixed order: a block's teams in shared memory, the blocks in a second
// small kernel.  Rows too wide for a block take several passes.
#pragma once
#include <algorithm>
#include <cmath>

#include "elem.cuh"
#include "kcommon.cuh"
#include "packed.cuh"
#include "train.h"

namespace ibwd {
namespace {

constexpr int kThreads = 256;     // block of several teams, and of the kernels for wide rows
constexpr int kMaxTeam = 512;     // threads of a block that is one team
constexpr int kElems = 16;        // elements of a row a thread holds at most
// Threads of an SM by the elements each holds (64 to 128 registers).  Shorter
// rows take eight elements a thread, which leaves more warps: fp32 rows of up
// to 2048 (14648x2047: 41 us, with sixteen 50), 16-bit ones of under 1024
// (46152x650: 32 against 35; 14648x2048: 25 against 18).  The backward pass
// of shifted fp32 rows gains from sixteen at over 1024 already (14648x2047: 75
// against 67).
constexpr int kFewElems = 8;
template <typename T>
constexpr int kFewWidth = kThreads * kFewElems / (sizeof(T) == 4 ? 1 : 2) - (sizeof(T) == 4 ? 0 : 1);
constexpr int fwd_per_sm(int elems, int team, bool late) {
  return elems <= kFewElems || late ? 1024 : team == 0 ? 768 : 512;
}
constexpr int bwd_per_sm(int elems, bool late) { return late ? 1024 : elems > kFewElems ? 512 : 768; }
constexpr int kMaxTeamWidth = kMaxTeam * kElems;
// Wider rows: teams of up to 1024 threads with 64 registers each, two blocks
// an SM up to 8192 elements.  The weights wait in shared memory beside the
// ring, in the order of their use, and a row's place in the ring is fetched
// into as soon as it was read.  From 4097 elements on this beats 512 threads
// of 128 registers, of which an SM holds but one block, in the forward pass of
// 16-bit rows (8192x4104: 44 us against 30; x8192: 54 against 52) and shifted
// fp32 ones (8192x5003: 68 against 59; but 4096x8192, not shifted, 44 against
// 49), and in the backward pass of fp32 rows (8192x5120: 112 against 90; but
// 8192x8192 in bf16, where the weights are read twice for every two bytes, 79
// against 96).  Beyond 8192 it is the only one (weights from L1 instead:
// 8192x12288 in bf16 100 us against 86, shifted 278 against 112).
constexpr int kLateTeam = 1024;
constexpr int kMaxLateWidth = kLateTeam * kElems;
// Rows of a team in flight or in work: four, or as many of the widest rows as
// 192 KB of shared memory hold (beside the weights).
constexpr int ring_stages(int maxt, int row_bytes, int weights) {
  return maxt > kMaxTeam ? std::min(4, (192 * 1024 - weights * 4 * kMaxLateWidth) / (kLateTeam * row_bytes))
                         : std::min(4, 192 * 1024 / (kMaxTeam * row_bytes));
}

// VEC consecutive elements as they lie in memory.
template <typename T, int VEC>
struct Chunk {
  static constexpr int kBytes = VEC * (int)sizeof(T);
  alignas(kBytes < 16 ? kBytes : 16) T e[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(e)[i] = ld_stream(reinterpret_cast<const uint4*>(p) + i);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(e) = *reinterpret_cast<const uint32_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        st_stream(reinterpret_cast<uint4*>(p) + i, reinterpret_cast<const uint4*>(e)[i]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(e);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = e[i];
    }
  }
};

// A thread's slots in a ring of rows in shared memory: K chunks a row, each in
// pieces of at most 16 bytes that lie side by side for neighbouring threads.
// The thread that copies a chunk is the only one that reads it.  A copy takes
// 4, 8 or 16 bytes; single 16-bit elements have none.
template <typename T, int VEC, int K>
struct Ring {
  static constexpr int kBytes = VEC * (int)sizeof(T);
  static constexpr bool kAsync = kBytes >= 4;
  static constexpr int kPiece = kBytes < 16 ? kBytes : 16;
  static constexpr int kRow = K * kBytes;  // bytes of a thread and row
  uint32_t base;                           // of this thread
  uint32_t pitch;                          // bytes between the pieces of a thread
  __device__ Ring(unsigned char* smem, int t, int threads)
      : base(smem_u32(smem) + t * kPiece), pitch(threads * kPiece) {}
  __device__ __forceinline__ void copy(int stage, int k, const T* src) const {
#pragma unroll
    for (int i = 0; i < kBytes / kPiece; ++i) {
      const uint32_t dst = base + ((stage * K + k) * (kBytes / kPiece) + i) * pitch;
      const char* from = reinterpret_cast<const char*>(src) + i * kPiece;
      if constexpr (kPiece == 16)
        cp_async16(dst, from, 16);
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(from), "n"(kPiece) : "memory");
    }
  }
  __device__ __forceinline__ void read(int stage, int k, Chunk<T, VEC>& c) const {
#pragma unroll
    for (int i = 0; i < kBytes / kPiece; ++i) {
      const uint32_t src = base + ((stage * K + k) * (kBytes / kPiece) + i) * pitch;
      if constexpr (kPiece == 16) {
        reinterpret_cast<uint4*>(c.e)[i] = ld_shared_v4(src);
      } else if constexpr (kPiece == 8) {
        uint2 v;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(src));
        *reinterpret_cast<uint2*>(c.e) = v;
      } else {
        uint32_t v;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(src));
        *reinterpret_cast<uint32_t*>(c.e) = v;
      }
    }
  }
};

// A thread's slots for its weights of a row in shared memory, in pieces of 16
// bytes that lie side by side for neighbouring threads.
template <int VEC>
struct WeightSlots {
  static constexpr int kPieces = VEC / 4;
  uint32_t base, pitch;
  __device__ WeightSlots(unsigned char* smem, int t, int threads) : base(smem_u32(smem) + t * 16), pitch(threads * 16) {}
  __device__ __forceinline__ void put(int k, const float2 (&w)[VEC / 2]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(base + (k * kPieces + i) * pitch), "f"(w[2 * i].x),
                   "f"(w[2 * i].y), "f"(w[2 * i + 1].x), "f"(w[2 * i + 1].y)
                   : "memory");
  }
  __device__ __forceinline__ void get(int k, float2 (&w)[VEC / 2]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(w[2 * i].x), "=f"(w[2 * i].y), "=f"(w[2 * i + 1].x), "=f"(w[2 * i + 1].y)
                   : "r"(base + (k * kPieces + i) * pitch));
  }
};

// gamma / beta element n as fp32: fp32 or the type of x.
template <typename T>
__device__ __forceinline__ float weight(const void* w, int n, bool f32, float none) {
  if (w == nullptr) return none;
  return f32 ? static_cast<const float*>(w)[n] : to_f32(static_cast<const T*>(w)[n]);
}

// gamma / beta of this thread's elements as pairs: K chunks of VEC, T chunks
// apart, from column `head` on; `none` without a vector and 0 beyond the row.
template <typename TX, int VEC, int K>
__device__ __forceinline__ void weights(float2 (&out)[K * VEC / 2], const void* w, bool f32, float none, int t, int T,
                                        int nvec, int head = 0) {
  const bool wide = VEC >= 4 && f32 && w != nullptr && ((reinterpret_cast<uintptr_t>(w) + 4 * head) & 15) == 0;
  if (wide) {
#pragma unroll
    for (int i = 0; i < K * VEC / 4; ++i) {
      const int j = t + 4 * i / VEC * T;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < nvec) v = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + head + j * VEC + 4 * i % VEC);
      out[2 * i] = make_float2(v.x, v.y);
      out[2 * i + 1] = make_float2(v.z, v.w);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < K * VEC / 2; ++i) {
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = 2 * i + h, j = t + e / VEC * T;
      v[h] = j < nvec ? weight<TX>(w, head + j * VEC + e % VEC, f32, none) : 0.f;
    }
    out[i] = make_float2(v[0], v[1]);
  }
}

// Elements 2i and 2i + 1 of a chunk list as fp32, and back.
template <typename T, int VEC, int K>
__device__ __forceinline__ float2 pair_of(const Chunk<T, VEC> (&c)[K], int i) {
  if constexpr (VEC == 1) {
    return make_float2(to_f32(c[2 * i].e[0]), to_f32(c[2 * i + 1].e[0]));
  } else {
    const T* e = &c[2 * i / VEC].e[2 * i % VEC];
    if constexpr (sizeof(T) == 4) {
      return make_float2(to_f32(e[0]), to_f32(e[1]));
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(e);
      return unpack2(w, T{});
    }
  }
}
template <typename T, int VEC, int K>
__device__ __forceinline__ void set_pair(Chunk<T, VEC> (&c)[K], int i, float2 v) {
  if constexpr (VEC == 1) {
    c[2 * i].e[0] = from_f32<T>(v.x);
    c[2 * i + 1].e[0] = from_f32<T>(v.y);
  } else {
    T* e = &c[2 * i / VEC].e[2 * i % VEC];
    if constexpr (sizeof(T) == 4) {
      e[0] = v.x;
      e[1] = v.y;
    } else {
      *reinterpret_cast<uint32_t*>(e) = pack2_of(v, T{});
    }
  }
}

// How a team's rows split: `nvec` vectors from element `head` on, and (SHIFT)
// the single elements before and after them, one a thread.  The rows of a
// team lie a multiple of eight rows apart, so they all begin at the same place
// of a 16-byte block, whatever their stride.
template <bool SHIFT>
struct Split {
  int head = 0, nvec, single = 0;
  bool has_single = false;
  template <typename T>
  __device__ Split(const T* row, int N, int vec, int t) {
    if (SHIFT) {
      head = min(N, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T));
      nvec = (N - head) / vec;
      has_single = t < N - nvec * vec;
      single = t < head ? t : t + nvec * vec;
    } else {
      nvec = N / vec;
    }
  }
};

// Columns of a group's sums in the workspace: 16-byte pieces.
__host__ __device__ constexpr int part_pitch(int N) { return (N + 3) / 4 * 4; }

// Two consecutive column sums at an even column: 8 bytes where the row of
// sums begins on an even one, too.
__device__ __forceinline__ void put_pair(float* p, float2 v) {
  if ((reinterpret_cast<uintptr_t>(p) & 7) == 0) {
    *reinterpret_cast<float2*>(p) = v;
  } else {
    p[0] = v.x;
    p[1] = v.y;
  }
}

// Sums of K values over a team, the same bits in each of its threads.  TEAM
// lanes of a warp, or 0 for the block: then `stage` holds 2 * K * 32 floats,
// zero beyond the block's warps and used in turn (`turn` flips), so one
// barrier a call is enough.
template <int TEAM, int K>
__device__ __forceinline__ void team_sums(float (&v)[K], float* stage, int& turn) {
#pragma unroll
  for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (TEAM == 0) {
    float* s = stage + turn * 32 * K;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[k * 32 + (threadIdx.x >> 5)] = v[k];
    __syncthreads();
    float4 f[K];
#pragma unroll
    for (int k = 0; k < K; ++k) f[k] = *reinterpret_cast<const float4*>(s + k * 32);
    for (int w = 4; w < (int)(blockDim.x >> 5); w += 4)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float4 o = *reinterpret_cast<const float4*>(s + k * 32 + w);
        f[k].x += o.x;
        f[k].y += o.y;
        f[k].z += o.z;
        f[k].w += o.w;
      }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = (f[k].x + f[k].y) + (f[k].z + f[k].w);
  }
}

// s / n given 1 / n, to the last bit but one (a constant row gets its value):
// the remainder of the product is added back (an infinity has none).
__device__ __forceinline__ float over_n(float s, float n, float inv_n) {
  const float q = s * inv_n;
  return isinf(q) ? q : fmaf(fmaf(-q, n, s), inv_n, q);
}

template <typename TX, typename TY, int VEC, int K, int TEAM, int MAXT, bool SHIFT>
__global__ void __launch_bounds__(MAXT, fwd_per_sm(VEC * K, TEAM, MAXT > kMaxTeam) / MAXT) norm_fwd_team(NormFwdArgs a) {
  constexpr bool kLate = MAXT > kMaxTeam;  // weights come from shared memory for each row
  constexpr int kStages = ring_stages(MAXT, VEC * K * (int)sizeof(TX), 2);
  constexpr int kAhead = kLate ? kStages : kStages - 1;  // rows fetched before the loop
  extern __shared__ __align__(16) unsigned char smem[];  // the ring
  __shared__ __align__(16) float stage[64];
  constexpr int TPB = TEAM ? kThreads / (TEAM ? TEAM : 1) : 1;
  constexpr int P = K * VEC / 2;  // pairs a thread
  const int team = TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0;
  const int t = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x, T = TEAM ? TEAM : blockDim.x;
  const float inv_n = 1.f / a.N;
  if (TEAM == 0)
    for (int i = threadIdx.x; i < 64; i += blockDim.x) stage[i] = 0.f;
  if (TEAM == 0) __syncthreads();
  const long long step = (long long)gridDim.x * TPB;
  const long long first = (long long)blockIdx.x * TPB + team;
  const TX* xr = static_cast<const TX*>(a.x) + first * a.x_stride;  // of the row to fetch
  const long long x_step = step * a.x_stride, y_step = step * a.y_stride;
  TY* yr = static_cast<TY*>(a.y) + first * a.y_stride;
  const Split<SHIFT> sp(xr, a.N, VEC, t);
  const int nvec = sp.nvec;
  const TX* x1 = xr + sp.single;
  TY* y1 = yr + sp.single;
  xr += sp.head + t * VEC;
  yr += sp.head + t * VEC;
  float2 g[kLate ? 1 : P], b[kLate ? 1 : P];
  const WeightSlots<VEC> gs(smem + kStages * K * VEC * sizeof(TX) * T, t, T);
  const WeightSlots<VEC> bs(smem + K * VEC * (kStages * sizeof(TX) + sizeof(float)) * T, t, T);
  if constexpr (!kLate) {
    weights<TX, VEC, K>(g, a.gamma, a.w_type == 0, 1.f, t, T, nvec, sp.head);
    weights<TX, VEC, K>(b, a.beta, a.w_type == 0, 0.f, t, T, nvec, sp.head);
  } else {
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
      float2 w[VEC / 2];
      weights<TX, VEC, 1>(w, a.gamma, a.w_type == 0, 1.f, t + k * T, T, nvec, sp.head);
      gs.put(k, w);
      weights<TX, VEC, 1>(w, a.beta, a.w_type == 0, 0.f, t + k * T, T, nvec, sp.head);
      bs.put(k, w);
    }
  }
  float g1 = 0.f, b1 = 0.f, next1 = 0.f;  // of the thread's single element
  if (SHIFT && sp.has_single) {
    g1 = weight<TX>(a.gamma, sp.single, a.w_type == 0, 1.f);
    b1 = weight<TX>(a.beta, sp.single, a.w_type == 0, 0.f);
    if (first < a.rows) next1 = to_f32(*x1);
  }
  using XRing = Ring<TX, VEC, K>;
  const XRing ring(smem, threadIdx.x, blockDim.x);
  Chunk<TX, VEC> cur[K] = {};  // (zero where a thread has no element)
  auto fetch = [&](int slot, bool on) {
    if (XRing::kAsync && on)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k * T < nvec) ring.copy(slot, k, xr + k * T * VEC);
    xr += x_step;
    cp_async_commit();
  };
  int turn = 0, slot = 0;
  if (XRing::kAsync)
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i, first + i * step < a.rows);
  // (a block's teams leave together: their rows differ by less than a step)
  for (long long r = first; r - team < a.rows; r += step) {
    const bool on = r < a.rows;
    if (XRing::kAsync) {
      if (!kLate) fetch(slot == 0 ? kStages - 1 : slot - 1, r + (kStages - 1) * step < a.rows);
      cp_async_wait<kStages - 1>();
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (on && t + k * T < nvec) {
        if constexpr (XRing::kAsync)
          ring.read(slot, k, cur[k]);
        else
          cur[k].load(xr + k * T * VEC);
      }
    if (!XRing::kAsync) xr += x_step;
    if (kLate && XRing::kAsync) fetch(slot, r + kStages * step < a.rows);  // into the place just read
    slot = slot == kStages - 1 ? 0 : slot + 1;
    float v1 = next1;
    if (SHIFT) {
      x1 += x_step;
      if (sp.has_single && r + step < a.rows) next1 = to_f32(*x1);
    }
    float2 v[kLate ? 1 : P], sum = both(0.f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 e = pair_of(cur, i);
      if (!kLate) v[kLate ? 0 : i] = e;
      sum = add2(sum, e);
    }
    float s[1] = {sum.x + sum.y};
    if (SHIFT && sp.has_single) s[0] += v1;
    team_sums<TEAM>(s, stage, turn);
    const float mean = over_n(s[0], (float)a.N, inv_n);
    sum = both(0.f);
    // elements the thread does not have are left out of the squares
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 e = add2(kLate ? pair_of(cur, i) : v[kLate ? 0 : i], both(-mean));
      if (!kLate) v[kLate ? 0 : i] = e;
      if constexpr (VEC > 1) {
        if (t + 2 * i / VEC * T < nvec) sum = fma2(e, e, sum);
      } else {
        if (t + 2 * i * T < nvec) sum.x = fmaf(e.x, e.x, sum.x);
        if (t + (2 * i + 1) * T < nvec) sum.y = fmaf(e.y, e.y, sum.y);
      }
    }
    float q[1] = {sum.x + sum.y};
    if (SHIFT && sp.has_single) {
      v1 -= mean;
      q[0] = fmaf(v1, v1, q[0]);
    }
    team_sums<TEAM>(q, stage, turn);
    const float rstd = rsqrtf(fmaf(q[0], inv_n, a.eps));
    if (on) {
      if constexpr (!kLate) {
        Chunk<TY, VEC> o[K];
#pragma unroll
        for (int i = 0; i < P; ++i) set_pair(o, i, fma2(mul2(v[i], both(rstd)), g[i], b[i]));
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (t + k * T < nvec) o[k].store(yr + k * T * VEC);
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (t + k * T >= nvec) break;
          Chunk<TY, VEC> o[1];
          float2 gk[VEC / 2], bk[VEC / 2];
          gs.get(k, gk);
          bs.get(k, bk);
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float2 e = add2(pair_of(cur, k * VEC / 2 + i), both(-mean));
            set_pair(o, i, fma2(mul2(e, both(rstd)), gk[i], bk[i]));
          }
          o[0].store(yr + k * T * VEC);
        }
      }
      if (SHIFT && sp.has_single) *y1 = from_f32<TY>(fmaf(v1 * rstd, g1, b1));
      if (t == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
      }
    }
    yr += y_step;
    if (SHIFT) y1 += y_step;
  }
  cp_async_wait_all();
}

template <typename TX, typename TD, int VEC, int K, int TEAM, int MAXT, bool SHIFT>
__global__ void __launch_bounds__(MAXT, bwd_per_sm(VEC * K, MAXT > kMaxTeam) / MAXT) norm_bwd_team(NormBwdArgs a) {
  // weights come from shared memory, and x and dy twice from the ring, for each row
  constexpr bool kLate = MAXT > kMaxTeam;
  constexpr int kStages = ring_stages(MAXT, VEC * K * (int)(sizeof(TX) + sizeof(TD)), 1);
  constexpr int kAhead = kLate ? kStages : kStages - 1;  // rows fetched before the loop
  extern __shared__ __align__(16) unsigned char smem[];  // the rings of x and dy; at the end the teams' column sums
  __shared__ __align__(16) float stage[128];
  constexpr int TPB = TEAM ? kThreads / (TEAM ? TEAM : 1) : 1;
  constexpr int P = K * VEC / 2;  // pairs a thread
  const int team = TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0;
  const int t = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x, T = TEAM ? TEAM : blockDim.x;
  const float inv_n = 1.f / a.N;
  if (TEAM == 0)
    for (int i = threadIdx.x; i < 128; i += blockDim.x) stage[i] = 0.f;
  if (TEAM == 0) __syncthreads();
  const long long step = (long long)gridDim.x * TPB;
  const long long first = (long long)blockIdx.x * TPB + team;
  const TX* xr = static_cast<const TX*>(a.x) + first * a.x_stride;  // of the row to fetch
  const TD* dr = static_cast<const TD*>(a.dy) + first * a.dy_stride;
  TX* or_ = static_cast<TX*>(a.dx) + first * a.dx_stride;
  const long long x_step = step * a.x_stride, d_step = step * a.dy_stride, o_step = step * a.dx_stride;
  const Split<SHIFT> sp(xr, a.N, VEC, t);
  const int nvec = sp.nvec;
  const TX* x1 = xr + sp.single;
  const TD* d1 = dr + sp.single;
  TX* o1 = or_ + sp.single;
  xr += sp.head + t * VEC;
  dr += sp.head + t * VEC;
  or_ += sp.head + t * VEC;
  float2 g[kLate ? 1 : P], dg[P], db[P];
  const WeightSlots<VEC> gs(smem + kStages * K * VEC * (sizeof(TX) + sizeof(TD)) * T, t, T);
  if constexpr (!kLate) {
    weights<TX, VEC, K>(g, a.gamma, a.w_type == 0, 1.f, t, T, nvec, sp.head);
  } else {
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
      float2 w[VEC / 2];
      weights<TX, VEC, 1>(w, a.gamma, a.w_type == 0, 1.f, t + k * T, T, nvec, sp.head);
      gs.put(k, w);
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) dg[i] = db[i] = both(0.f);
  // of the thread's single element
  float g1 = 0.f, dg1 = 0.f, db1 = 0.f, next_x = 0.f, next_d = 0.f;
  if (SHIFT && sp.has_single) {
    g1 = weight<TX>(a.gamma, sp.single, a.w_type == 0, 1.f);
    if (first < a.rows) {
      next_x = to_f32(*x1);
      next_d = to_f32(*d1);
    }
  }
  using XRing = Ring<TX, VEC, K>;
  using DRing = Ring<TD, VEC, K>;
  constexpr bool kAsync = XRing::kAsync && DRing::kAsync;
  const XRing xring(smem, threadIdx.x, blockDim.x);
  const DRing dring(smem + kStages * XRing::kRow * blockDim.x, threadIdx.x, blockDim.x);
  // zero where a thread has no element: dy = 0 adds nothing to any sum
  Chunk<TX, VEC> cx[K] = {};
  Chunk<TD, VEC> cd[K] = {};
  auto fetch = [&](int slot, bool on) {
    if (kAsync && on)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k * T < nvec) {
          xring.copy(slot, k, xr + k * T * VEC);
          dring.copy(slot, k, dr + k * T * VEC);
        }
    xr += x_step;
    dr += d_step;
    cp_async_commit();
  };
  int turn = 0, slot = 0;
  if (kAsync)
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i, first + i * step < a.rows);
  float nm = 0.f, nr = 0.f;  // the next row's statistics
  if (first < a.rows) {
    nm = a.mean[first];
    nr = a.rstd[first];
  }
  for (long long r = first; r - team < a.rows; r += step) {
    const bool on = r < a.rows;
    const float cm = nm, cr = nr;
    if (r + step < a.rows) {
      nm = a.mean[r + step];
      nr = a.rstd[r + step];
    }
    if (kAsync) {
      if (!kLate) fetch(slot == 0 ? kStages - 1 : slot - 1, r + (kStages - 1) * step < a.rows);
      cp_async_wait<kStages - 1>();
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (!kLate && on && t + k * T < nvec) {
        if constexpr (kAsync) {
          xring.read(slot, k, cx[k]);
          dring.read(slot, k, cd[k]);
        } else {
          cx[k].load(xr + k * T * VEC);
          cd[k].load(dr + k * T * VEC);
        }
      }
    if (!kAsync) {
      xr += x_step;
      dr += d_step;
    }
    const int here = slot;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    const float vx = next_x, vd = next_d;
    if (SHIFT) {
      x1 += x_step;
      d1 += d_step;
      if (sp.has_single && r + step < a.rows) {
        next_x = to_f32(*x1);
        next_d = to_f32(*d1);
      }
    }
    float s[2] = {0.f, 0.f};
    if (on) {
      float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float2 gk[VEC > 1 ? VEC / 2 : 1];
        Chunk<TX, VEC> x[1];
        Chunk<TD, VEC> y[1];
        if constexpr (kLate) {
          if (t + k * T >= nvec) break;
          xring.read(here, k, x[0]);
          dring.read(here, k, y[0]);
          gs.get(k, gk);
        }
#pragma unroll
        for (int h = 0; h < VEC / 2 || (VEC == 1 && h < 1); ++h) {
          if (VEC == 1 && (k & 1)) continue;  // single elements pair up
          const int i = VEC == 1 ? k / 2 : k * VEC / 2 + h;
          const float2 xv = kLate ? pair_of(x, kLate ? h : 0) : pair_of(cx, i);
          const float2 dy = kLate ? pair_of(y, kLate ? h : 0) : pair_of(cd, i);
          const float2 xh = mul2(add2(xv, both(-cm)), both(cr));
          const float2 d = mul2(dy, kLate ? gk[h] : g[kLate ? 0 : i]);
          dg[i] = fma2(dy, xh, dg[i]);
          db[i] = add2(db[i], dy);
          s0 = add2(s0, d);
          s1 = fma2(d, xh, s1);
        }
      }
      s[0] = s0.x + s0.y;
      s[1] = s1.x + s1.y;
      if (SHIFT && sp.has_single) {
        const float xh = (vx - cm) * cr, d = vd * g1;
        dg1 = fmaf(vd, xh, dg1);
        db1 += vd;
        s[0] += d;
        s[1] = fmaf(d, xh, s[1]);
      }
    }
    team_sums<TEAM>(s, stage, turn);
    if (on) {
      const float ma = s[0] * inv_n, mb = s[1] * inv_n;
      if constexpr (!kLate) {
        Chunk<TX, VEC> o[K];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 xh = mul2(add2(pair_of(cx, i), both(-cm)), both(cr));
          const float2 d = fma2(pair_of(cd, i), g[i], both(-ma));
          set_pair(o, i, mul2(fma2(xh, both(-mb), d), both(cr)));
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (t + k * T < nvec) o[k].store(or_ + k * T * VEC);
      } else {
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
          if (t + k * T >= nvec) break;
          Chunk<TX, VEC> x[1], o[1];
          Chunk<TD, VEC> d[1];
          xring.read(here, k, x[0]);
          dring.read(here, k, d[0]);
          float2 gk[VEC / 2];
          gs.get(k, gk);
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float2 xh = mul2(add2(pair_of(x, i), both(-cm)), both(cr));
            set_pair(o, i, mul2(fma2(xh, both(-mb), fma2(pair_of(d, i), gk[i], both(-ma))), both(cr)));
          }
          o[0].store(or_ + k * T * VEC);
        }
      }
      if (SHIFT && sp.has_single) {
        const float xh = (vx - cm) * cr;
        *o1 = from_f32<TX>(cr * (fmaf(vd, g1, -ma) - xh * mb));
      }
    }
    if (kLate) fetch(here, r + kStages * step < a.rows);  // into the place just read
    if (SHIFT) o1 += o_step;
    or_ += o_step;
  }
  cp_async_wait_all();
  if (!a.dgamma && !a.dbeta) return;
  griddep_launch_dependents();  // the join's blocks come as these leave
  // The block's column sums: a group of part[groups][2][part_pitch] -- or,
  // where it is the only block, dgamma and dbeta.
  float* const out_g = gridDim.x > 1 ? a.part + (long long)blockIdx.x * 2 * part_pitch(a.N) : a.dgamma;
  float* const out_b = gridDim.x > 1 ? out_g + part_pitch(a.N) : a.dbeta;
  if constexpr (TEAM == 0) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int j = t + 2 * i / VEC * T, c = sp.head + j * VEC + 2 * i % VEC;
      if constexpr (VEC == 1) {
        if (j < nvec && out_g) out_g[c] = dg[i].x;
        if (j < nvec && out_b) out_b[c] = db[i].x;
        if (j + T < nvec && out_g) out_g[c + T] = dg[i].y;
        if (j + T < nvec && out_b) out_b[c + T] = db[i].y;
      } else {
        if (j < nvec && out_g) put_pair(out_g + c, dg[i]);
        if (j < nvec && out_b) put_pair(out_b + c, db[i]);
      }
    }
    if (SHIFT && sp.has_single) {
      if (out_g) out_g[sp.single] = dg1;
      if (out_b) out_b[sp.single] = db1;
    }
  } else {
    // the teams' sums side by side in shared memory, added in the teams' order
    float* const sums = reinterpret_cast<float*>(smem) + team * 2 * a.N;
    __syncthreads();  // the rings are done with
#pragma unroll
    for (int e = 0; e < 2 * P; ++e) {
      const int j = t + e / VEC * T, c = sp.head + j * VEC + e % VEC;
      if (j < nvec) {
        sums[c] = e & 1 ? dg[e / 2].y : dg[e / 2].x;
        sums[a.N + c] = e & 1 ? db[e / 2].y : db[e / 2].x;
      }
    }
    if (SHIFT && sp.has_single) {
      sums[sp.single] = dg1;
      sums[a.N + sp.single] = db1;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.N; c += kThreads) {
      float v = 0.f;
      for (int w = 0; w < TPB; ++w) v += reinterpret_cast<const float*>(smem)[w * 2 * a.N + c];
      if (c < a.N) {
        if (out_g) out_g[c] = v;
      } else if (out_b) {
        out_b[c - a.N] = v;
      }
    }
  }
}

// dgamma and dbeta from the groups' column sums [groups][2][part_pitch]: 32
// columns a block, eight threads by NT / 8 interleaved sums of groups, joined
// in order.
template <int NT>
__global__ void __launch_bounds__(NT) norm_bwd_join(const float* part, int groups, int N, float* dgamma,
                                                              float* dbeta) {
  constexpr int kSlices = NT / 8;
  __shared__ float s[kSlices][33];
  const int pitch = part_pitch(N);
  const int q = threadIdx.x & 7, w = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + 4 * q;
  griddep_wait();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < 2 * pitch) {
    const float* p = part + c;
#pragma unroll 4
    for (int i = w; i < groups; i += kSlices) {
      const float4 o = *reinterpret_cast<const float4*>(p + (long long)i * 2 * pitch);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
  }
  s[w][4 * q] = v.x;
  s[w][4 * q + 1] = v.y;
  s[w][4 * q + 2] = v.z;
  s[w][4 * q + 3] = v.w;
  __syncthreads();
  // a column (or several) a warp
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < 1024 / NT; ++e) {
    const int col = threadIdx.x / 32 + e * (NT / 32), cw = blockIdx.x * 32 + col;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices; i += 32) sum += s[i + lane][col];
    sum = warp_sum(sum);
    if (lane == 0) {
      if (cw < N) {
        if (dgamma) dgamma[cw] = sum;
      } else if (cw >= pitch && cw - pitch < N) {
        if (dbeta) dbeta[cw - pitch] = sum;
      }
    }
  }
}

// ------------------------------------------------------------- wide rows ---
// Any width and alignment: a block takes a row in three passes (two backward).

template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads) norm_fwd_wide(NormFwdArgs a) {
  __shared__ __align__(16) float stage[64];
  if (threadIdx.x < 64) stage[threadIdx.x] = 0.f;
  __syncthreads();
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const TX* x = static_cast<const TX*>(a.x) + r * a.x_stride;
    TY* y = static_cast<TY*>(a.y) + r * a.y_stride;
    float s[1] = {0.f};
    for (int n = threadIdx.x; n < a.N; n += kThreads) s[0] += to_f32(x[n]);
    team_sums<0>(s, stage, turn);
    const float mean = s[0] / a.N;
    float q[1] = {0.f};
    for (int n = threadIdx.x; n < a.N; n += kThreads) {
      const float d = to_f32(x[n]) - mean;
      q[0] += d * d;
    }
    team_sums<0>(q, stage, turn);
    const float rstd = 1.f / sqrtf(q[0] / a.N + a.eps);
    for (int n = threadIdx.x; n < a.N; n += kThreads)
      y[n] = from_f32<TY>((to_f32(x[n]) - mean) * rstd * weight<TX>(a.gamma, n, a.w_type == 0, 1.f) +
                          weight<TX>(a.beta, n, a.w_type == 0, 0.f));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

template <typename TX, typename TD>
__global__ void __launch_bounds__(kThreads) norm_bwd_wide(NormBwdArgs a) {
  __shared__ __align__(16) float stage[128];
  if (threadIdx.x < 128) stage[threadIdx.x] = 0.f;
  __syncthreads();
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const TX* x = static_cast<const TX*>(a.x) + r * a.x_stride;
    const TD* dy = static_cast<const TD*>(a.dy) + r * a.dy_stride;
    TX* dx = static_cast<TX*>(a.dx) + r * a.dx_stride;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s[2] = {0.f, 0.f};
    for (int n = threadIdx.x; n < a.N; n += kThreads) {
      const float d = to_f32(dy[n]) * weight<TX>(a.gamma, n, a.w_type == 0, 1.f);
      s[0] += d;
      s[1] += d * ((to_f32(x[n]) - mean) * rstd);
    }
    team_sums<0>(s, stage, turn);
    const float ma = s[0] / a.N, mb = s[1] / a.N;
    for (int n = threadIdx.x; n < a.N; n += kThreads) {
      const float xh = (to_f32(x[n]) - mean) * rstd;
      const float d = to_f32(dy[n]) * weight<TX>(a.gamma, n, a.w_type == 0, 1.f);
      dx[n] = from_f32<TX>(rstd * (d - ma - xh * mb));
    }
  }
}

// Column sums of row group blockIdx.y for the columns of blockIdx.x: 32
// columns by 8 interleaved rows a block, the eight joined in order.
template <typename TX, typename TD>
__global__ void __launch_bounds__(kThreads) norm_bwd_wide_columns(NormBwdArgs a, int group_rows) {
  __shared__ float sg[8][33], sb[8][33];
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + c;
  const long long r0 = (long long)blockIdx.y * group_rows;
  const long long r1 = min(a.rows, r0 + group_rows);
  float g = 0.f, b = 0.f;
  if (n < a.N)
    for (long long r = r0 + w; r < r1; r += 8) {
      const float d = to_f32(static_cast<const TD*>(a.dy)[r * a.dy_stride + n]);
      const float xh = (to_f32(static_cast<const TX*>(a.x)[r * a.x_stride + n]) - a.mean[r]) * a.rstd[r];
      g += d * xh;
      b += d;
    }
  sg[w][c] = g;
  sb[w][c] = b;
  __syncthreads();
  if (w == 0 && n < a.N) {
    g = b = 0.f;
    for (int i = 0; i < 8; ++i) {
      g += sg[i][c];
      b += sb[i][c];
    }
    a.part[((long long)blockIdx.y * 2) * part_pitch(a.N) + n] = g;
    a.part[((long long)blockIdx.y * 2 + 1) * part_pitch(a.N) + n] = b;
  }
}

// -------------------------------------------------------------- launches ---

constexpr int kMaxSms = 160;       // the workspace does not depend on the device
constexpr int kMaxWideGroups = 64;

// The shape of a team launch; teams_per_block 0: the block is the team.
struct TeamShape {
  int threads, blocks;
};

// All blocks resident: `per_sm` threads an SM.  Column sums: each block writes
// 8 N bytes that the join reads, so of R rows a block takes sqrt(R / 60) at
// least, or sqrt(R / 30) where its teams share them (64x16384 in bf16: 26.6 us
// with four rows a block, 17.5 with one; 8192x1024: 16.7 with seven, 13.7 with
// eleven).  shift: a team's rows lie a multiple of eight rows apart.
TeamShape team_shape(long long rows, int N, int elems, int teams_per_block, int per_sm, int num_sms, bool sums,
                     bool shift) {
  TeamShape s;
  s.threads = teams_per_block ? kThreads : std::max(32, ((N + elems - 1) / elems + 31) / 32 * 32);
  const int per_block = std::max(1, teams_per_block);
  const long long resident = (long long)std::min(num_sms, kMaxSms) * std::max(1, per_sm / s.threads);
  const long long all = (rows + per_block - 1) / per_block;  // blocks of one row a team
  s.blocks = (int)std::min(all, resident);
  if (sums) {
    const long long each = (long long)std::sqrt((double)all / (teams_per_block ? 30 : 60));
    if (each > 1) s.blocks = (int)std::min<long long>(s.blocks, (all + each - 1) / each);
  }
  if (shift) {
    // a multiple of eight, or one row a team
    if (s.blocks >= 8)
      s.blocks &= ~7;
    else
      s.blocks = (int)std::min<long long>(8, (rows + per_block - 1) / per_block);
  }
  return s;
}

// most: the shared memory of the kernel's largest launch; limit: of this kernel alone.
template <typename Args>
cudaError_t launch_team(void (*kern)(Args), const TeamShape& s, size_t smem, size_t most, std::atomic<size_t>* limit,
                        cudaStream_t st, const Args& a) {
  const cudaError_t e = raise_smem((const void*)kern, most, limit);
  if (e != cudaSuccess) return e;
  return launch_ex(kern, s.blocks, s.threads, smem, st, false, a);
}

bool aligned(const void* p, long long stride, int size, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * size % bytes == 0;
}

// Whether the vectors that begin x's rows' first whole 16-byte blocks begin
// aligned pieces of `bytes` in another matrix, too: for eight rows, after
// which every stride comes back to the same place.
bool shifts_alike(const void* x, long long x_stride, int x_size, const void* o, long long o_stride, int o_size,
                  int bytes) {
  for (int r = 0; r < 8; ++r) {
    const uintptr_t px = reinterpret_cast<uintptr_t>(x) + (uintptr_t)(r * x_stride * x_size);
    const uintptr_t head = ((16 - (px & 15)) & 15) / x_size;
    if ((reinterpret_cast<uintptr_t>(o) + (uintptr_t)(r * o_stride + (long long)head) * o_size) % bytes) return false;
  }
  return true;
}

template <typename TX, typename TY, int VEC, int E, int TEAM, int MAXT, bool SHIFT>
cudaError_t fwd_team(const NormFwdArgs& a, cudaStream_t st) {
  constexpr int K = E / VEC;
  const TeamShape s = team_shape(a.rows, a.N, E, TEAM ? kThreads / (TEAM ? TEAM : 1) : 0, fwd_per_sm(E, TEAM, MAXT > kMaxTeam), a.num_sms,
                                 false, SHIFT);
  using XRing = Ring<TX, VEC, K>;
  constexpr int stages = ring_stages(MAXT, XRing::kRow, 2);
  constexpr size_t each = (XRing::kAsync ? (size_t)stages * XRing::kRow : 0) + (MAXT > kMaxTeam ? 8 * E : 0);
  static std::atomic<size_t> limit[64];
  return launch_team(norm_fwd_team<TX, TY, VEC, K, TEAM, MAXT, SHIFT>, s, each * s.threads, each * MAXT, limit, st, a);
}

// Rows by 16-byte vectors of x, all aligned or (SHIFT) all of them shifted.
template <typename TX, typename TY, bool SHIFT>
cudaError_t fwd_vectors(const NormFwdArgs& a, cudaStream_t st) {
  constexpr int V = kVec<TX>;
  if (!SHIFT) {
    if (a.N <= 8 * V) return fwd_team<TX, TY, V, V, 8, kThreads, false>(a, st);
    if (a.N <= 16 * V) return fwd_team<TX, TY, V, V, 16, kThreads, false>(a, st);
    if (a.N <= 32 * V) return fwd_team<TX, TY, V, V, 32, kThreads, false>(a, st);
  }
  if (a.N <= 32 * kElems) return fwd_team<TX, TY, V, kElems, 32, kThreads, SHIFT>(a, st);
  if (a.N <= kFewWidth<TX>) return fwd_team<TX, TY, V, kFewElems, 0, kThreads, SHIFT>(a, st);
  if (a.N <= kThreads * kElems) return fwd_team<TX, TY, V, kElems, 0, kThreads, SHIFT>(a, st);
  if constexpr (sizeof(TX) == 4 && !SHIFT)
    if (a.N <= kMaxTeamWidth) return fwd_team<TX, TY, V, kElems, 0, kMaxTeam, SHIFT>(a, st);
  return fwd_team<TX, TY, V, kElems, 0, kLateTeam, SHIFT>(a, st);
}

template <typename TX, typename TY>
cudaError_t norm_fwd(const NormFwdArgs& a, cudaStream_t st) {
  constexpr int V = kVec<TX>, xs = (int)sizeof(TX), ys = (int)sizeof(TY);
  if (a.N <= kMaxLateWidth) {
    if (a.N % V == 0 && aligned(a.x, a.x_stride, xs, 16) && aligned(a.y, a.y_stride, ys, V * ys))
      return fwd_vectors<TX, TY, false>(a, st);
    if (shifts_alike(a.x, a.x_stride, xs, a.y, a.y_stride, ys, V * ys)) return fwd_vectors<TX, TY, true>(a, st);
  }
  if (a.N <= 32 * kElems) return fwd_team<TX, TY, 1, kElems, 32, kThreads, false>(a, st);
  if (a.N <= kMaxTeamWidth) return fwd_team<TX, TY, 1, kElems, 0, kMaxTeam, false>(a, st);
  return launch_ex(norm_fwd_wide<TX, TY>, (int)std::min<long long>(a.rows, 8LL * a.num_sms), kThreads, 0, st, false, a);
}

cudaError_t join_sums(const NormBwdArgs& a, int groups, cudaStream_t st) {
  // two groups a thread or more, and 256 threads or more (64x16384: 17.5 us by
  // 256 threads, 22 by 1024; 8192x1024, 745 groups: 20 and 14)
  const auto join = [&](auto* kern, int threads) {
    return launch_ex(kern, (2 * part_pitch(a.N) + 31) / 32, threads, 0, st, true, (const float*)a.part, groups, a.N,
                     a.dgamma, a.dbeta);
  };
  return groups >= 256   ? join(norm_bwd_join<1024>, 1024)
         : groups >= 128 ? join(norm_bwd_join<512>, 512)
                         : join(norm_bwd_join<256>, 256);
}

template <typename TX, typename TD, int VEC, int E, int TEAM, int MAXT, bool SHIFT>
cudaError_t bwd_team(const NormBwdArgs& a, cudaStream_t st) {
  constexpr int K = E / VEC;
  const bool sums = a.dgamma || a.dbeta;
  const TeamShape s = team_shape(a.rows, a.N, E, TEAM ? kThreads / (TEAM ? TEAM : 1) : 0, bwd_per_sm(E, MAXT > kMaxTeam), a.num_sms,
                                 sums, SHIFT);
  using XRing = Ring<TX, VEC, K>;
  using DRing = Ring<TD, VEC, K>;
  constexpr int stages = ring_stages(MAXT, XRing::kRow + DRing::kRow, 1);
  constexpr size_t each = XRing::kAsync && DRing::kAsync
                              ? (size_t)stages * (XRing::kRow + DRing::kRow) + (MAXT > kMaxTeam ? 4 * E : 0)
                              : 0;
  // the teams' column sums: rows of up to TEAM E elements
  constexpr size_t team_sums = TEAM ? kThreads / (TEAM ? TEAM : 1) * 2 * sizeof(float) : 0;
  const size_t smem = std::max(each * s.threads, sums ? team_sums * a.N : 0);
  constexpr size_t most = std::max(each * MAXT, team_sums * TEAM * E);
  static std::atomic<size_t> limit[64];
  cudaError_t e = launch_team(norm_bwd_team<TX, TD, VEC, K, TEAM, MAXT, SHIFT>, s, smem, most, limit, st, a);
  if (e == cudaSuccess && sums && s.blocks > 1) e = join_sums(a, s.blocks, st);
  return e;
}

template <typename TX, typename TD, bool SHIFT>
cudaError_t bwd_vectors(const NormBwdArgs& a, cudaStream_t st) {
  constexpr int V = kVec<TX>;
  if (!SHIFT) {
    if (a.N <= 8 * V) return bwd_team<TX, TD, V, V, 8, kThreads, false>(a, st);
    if (a.N <= 16 * V) return bwd_team<TX, TD, V, V, 16, kThreads, false>(a, st);
    if (a.N <= 32 * V) return bwd_team<TX, TD, V, V, 32, kThreads, false>(a, st);
  }
  if (a.N <= 32 * kElems) return bwd_team<TX, TD, V, kElems, 32, kThreads, SHIFT>(a, st);
  if (a.N <= kFewWidth<TX> / (SHIFT && sizeof(TX) == 4 ? 2 : 1)) return bwd_team<TX, TD, V, kFewElems, 0, kThreads, SHIFT>(a, st);
  if (a.N <= kThreads * kElems) return bwd_team<TX, TD, V, kElems, 0, kThreads, SHIFT>(a, st);
  if constexpr (sizeof(TX) == 2)
    if (a.N <= kMaxTeamWidth) return bwd_team<TX, TD, V, kElems, 0, kMaxTeam, SHIFT>(a, st);
  return bwd_team<TX, TD, V, kElems, 0, kLateTeam, SHIFT>(a, st);
}

template <typename TX, typename TD>
cudaError_t norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  constexpr int V = kVec<TX>, xs = (int)sizeof(TX), ds = (int)sizeof(TD);
  const bool sums = a.dgamma || a.dbeta;
  if (!a.rows) {
    cudaError_t e = cudaSuccess;
    if (a.dgamma) e = cudaMemsetAsync(a.dgamma, 0, a.N * sizeof(float), st);
    if (a.dbeta && e == cudaSuccess) e = cudaMemsetAsync(a.dbeta, 0, a.N * sizeof(float), st);
    return e;
  }
  if (a.N <= kMaxLateWidth) {
    constexpr int piece = std::min(16, V * ds);
    if (a.N % V == 0 && aligned(a.x, a.x_stride, xs, 16) && aligned(a.dx, a.dx_stride, xs, 16) &&
        aligned(a.dy, a.dy_stride, ds, piece))
      return bwd_vectors<TX, TD, false>(a, st);
    if (shifts_alike(a.x, a.x_stride, xs, a.dx, a.dx_stride, xs, 16) &&
        shifts_alike(a.x, a.x_stride, xs, a.dy, a.dy_stride, ds, piece))
      return bwd_vectors<TX, TD, true>(a, st);
  }
  if (a.N <= 32 * kElems) return bwd_team<TX, TD, 1, kElems, 32, kThreads, false>(a, st);
  if (a.N <= kMaxTeamWidth) return bwd_team<TX, TD, 1, kElems, 0, kMaxTeam, false>(a, st);
  if (sums) {  // before the rows: dx may be x or dy
    const int groups = (int)std::min<long long>(kMaxWideGroups, (a.rows + 31) / 32);
    const int group_rows = (int)((a.rows + groups - 1) / groups);
    cudaError_t e = launch_ex(norm_bwd_wide_columns<TX, TD>, dim3((a.N + 31) / 32, groups), kThreads, 0, st, false, a,
                              group_rows);
    if (e == cudaSuccess) e = join_sums(a, groups, st);
    if (e != cudaSuccess) return e;
  }
  return launch_ex(norm_bwd_wide<TX, TD>, (int)std::min<long long>(a.rows, 8LL * a.num_sms), kThreads, 0, st, false, a);
}

}  // namespace
}  // namespace ibwd
