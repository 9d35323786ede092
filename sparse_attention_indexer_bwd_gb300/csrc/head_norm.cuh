// Norm of each head of queries and keys with the position rotation in the
// same pass, and its backward pass.
//
//   xh = (x - mean) rstd (layer), x rstd (rms) or x,   z = xh gamma + beta,
//   y_a = z_a cos t - z_b sin t,   y_b = z_b cos t + z_a sin t
// for the pairs (a, b) of the rotated dimensions, t = position * freq; backward
// dz is dy turned by -t, d = dz gamma, and
//   dx = rstd (d - [layer: sum(d)/D] - xh sum(d xh)/D),
//   dgamma = sum dz xh,  dbeta = sum dz over tokens and heads.
// The backward pass takes its statistics from x again, which it has to read
// anyway: nothing has to be kept from the forward pass.
//
// Angles: a frequency becomes a 64-bit fraction of a turn, so that its product
// with a position, modulo 2^64, is the angle modulo a turn without rounding:
// far positions lose nothing. A quarter turn is taken off in integers, what is
// left goes through sincospi on [-1/4, 1/4].
#pragma once
#include "elem.cuh"
#include "head_norm.h"
#include "indexer_train.h"
#include "kcommon.cuh"
#include "packed.cuh"
#include "train.h"

#include <atomic>
#include <climits>
#include <type_traits>

namespace ibwd {

constexpr int kHeadThreads = 256;
constexpr int kHeadAngles = 2048;  // of a block's table at most: a group's tokens times the pairs
// In front of a ring of rows: the table, and the weights of 16 lanes that are wide. (A backward pass's column sums, 16 KB for
// heads of 256, take the table's place.)
constexpr size_t kHeadFront = kHeadAngles * 8 + 16 * 64;

__device__ __forceinline__ float weight_at(const void* w, int type, int i) {
  if (type == IBWD_F32) return static_cast<const float*>(w)[i];
  if (type == IBWD_BF16) return to_f32(static_cast<const __nv_bfloat16*>(w)[i]);
  return to_f32(static_cast<const __half*>(w)[i]);
}

// N elements side by side, as they lie in memory: 8, 16 or 32 bytes.
template <typename T, int N>
struct Part {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  // A thread's slot in shared memory lies in words of kChunk bytes, the threads' side by side.
  static constexpr int kChunk = kWords == 2 ? 8 : 16, kChunks = kWords * 4 / kChunk, kStride = kChunk * kHeadThreads;
  __device__ static void copy(uint32_t slot, const T* p) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const T* from = p + i * kChunk / (int)sizeof(T);
      if constexpr (kChunk == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot + i * kStride), "l"(from) : "memory");
      else
        cp_async16(slot + i * kStride, from, 16);
    }
  }
  __device__ void take(uint32_t slot) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if constexpr (kChunk == 8)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(slot) : "memory");
      else
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(slot + i * kStride)
                     : "memory");
    }
  }
  __device__ static void clear(uint32_t slot) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int k = 0; k < kChunk; k += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(slot + i * kStride + k), "r"(0) : "memory");
  }
  __device__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 a = unpack2(w[i], T{});
        v[2 * i] = a.x, v[2 * i + 1] = a.y;
      }
    }
  }
  __device__ static void store(T* p, const float (&v)[N]) {
    uint32_t x[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4)
        x[i] = __float_as_uint(v[i]);
      else
        x[i] = pack2_of(make_float2(v[2 * i], v[2 * i + 1]), T{});
    }
    if constexpr (kWords == 2) {
      asm volatile("st.global.L1::no_allocate.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(x[0]), "r"(x[1]) : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) st_stream(p + i * 4 / (int)sizeof(T), make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]));
    }
  }
};

// A lane's 2 N elements of a row: partners a_i and b_i of N pairs, packed
// by twos (two fp32 an instruction).
template <int N>
struct Pairs {
  float2 a[N / 2], b[N / 2];
};
// INTER: parts (a0 b0 a1 b1 ..) of the row's first half and of its second; otherwise (a0 a1 ..) and (b0 b1 ..).
template <bool INTER, int N>
__device__ __forceinline__ Pairs<N> paired(const float (&x)[N], const float (&y)[N]) {
  Pairs<N> e;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (INTER) {
      const float* v = i < N / 4 ? x + 4 * i : y + 4 * (i - N / 4);
      e.a[i] = make_float2(v[0], v[2]), e.b[i] = make_float2(v[1], v[3]);
    } else {
      e.a[i] = make_float2(x[2 * i], x[2 * i + 1]), e.b[i] = make_float2(y[2 * i], y[2 * i + 1]);
    }
  }
  return e;
}
template <bool INTER, int N>
__device__ __forceinline__ void apart(const Pairs<N>& e, float (&x)[N], float (&y)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (INTER) {
      float* v = i < N / 4 ? x + 4 * i : y + 4 * (i - N / 4);
      v[0] = e.a[i].x, v[1] = e.b[i].x, v[2] = e.a[i].y, v[3] = e.b[i].y;
    } else {
      x[2 * i] = e.a[i].x, x[2 * i + 1] = e.a[i].y, y[2 * i] = e.b[i].x, y[2 * i + 1] = e.b[i].y;
    }
  }
}
template <int N>
__device__ __forceinline__ float total(const Pairs<N>& v) {
  float2 t = add2(v.a[0], v.b[0]);
#pragma unroll
  for (int i = 1; i < N / 2; ++i) t = add2(t, add2(v.a[i], v.b[i]));
  return t.x + t.y;
}
template <int N>
__device__ __forceinline__ float product(const Pairs<N>& v, const Pairs<N>& w) {
  float2 t = mul2(v.a[0], w.a[0]);
#pragma unroll
  for (int i = 1; i < N / 2; ++i) t = fma2(v.a[i], w.a[i], t);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) t = fma2(v.b[i], w.b[i], t);
  return t.x + t.y;
}
template <int N>
__device__ __forceinline__ void shift(Pairs<N>& v, float by) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    v.a[i] = add2(v.a[i], both(by));
    v.b[i] = add2(v.b[i], both(by));
  }
}

// Sums over a group of L lanes, in every one of them.
template <int L, int U>
__device__ __forceinline__ void group_sums(float (&v)[U]) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
}

// The rotation of a tile's tokens in shared memory: [tokens][pairs] cosines,
// then sines, filled by the whole block; every head of a token takes them from
// there, so that their 40 instructions a pair are spent once a token and
// operand (per head they would be three times the norm's). A thread has one
// pair, whose frequency stays in registers.
struct Turns {
  float* cs;
  float* sn;
  unsigned long long freq = 0;  // fraction of a turn
  int pair = 0, token = 0, step = 1, axis = -1;

  __device__ Turns(unsigned char* smem, const HeadArgs& a, int tokens) {
    cs = reinterpret_cast<float*>(smem);
    sn = cs + tokens * a.pairs;
    if (!a.pairs) return;
    step = kHeadThreads / a.pairs;
    token = threadIdx.x / a.pairs;
    pair = threadIdx.x - token * a.pairs;
    if (token >= step) return;
    const double f = a.freq64 ? static_cast<const double*>(a.freq)[pair] : (double)static_cast<const float*>(a.freq)[pair];
    const double turns = f * 0.15915494309189533577;  // 1 / 2 pi
    // modulo a turn by its bits: fp64's operations are slow here
    const long long bits = __double_as_longlong(turns);
    const unsigned long long m = (bits & 0xFFFFFFFFFFFFFll) | 0x10000000000000ll;
    const int by = (int)(bits >> 52 & 2047) - 1011;  // m 2^by in 2^-64 turns
    freq = by >= 64 || by <= -64 ? 0 : by >= 0 ? m << by : m >> -by;
    if (bits < 0) freq = 0 - freq;
    axis = a.axis_of ? a.axis_of[pair] : 0;
  }
  __device__ void fill(const HeadArgs& a, long long first, int tokens) const {
    if (!a.pairs || token >= step) return;
    const int end = (int)min((long long)tokens, a.tokens - first);
    for (int t = token; t < end; t += step) {
      float s = 0.f, c = 1.f;
      // an axis that does not exist turns nothing
      if ((unsigned)axis < (unsigned)a.axes) {
        const long long at = axis * a.axis_stride + first + t;
        const long long pos = a.positions64 ? static_cast<const long long*>(a.positions)[at]
                                            : (long long)static_cast<const int*>(a.positions)[at];
        const int turn = (int)((freq * (unsigned long long)pos) >> 32);  // 2^-32 turns
        const int quarter = (int)(((unsigned)turn + 0x20000000u) >> 30);
        const float r = (float)(int)((unsigned)turn - ((unsigned)quarter << 30)) * 0x1p-31f;  // half turns
        float sr, cr;
        sincospif(r, &sr, &cr);
        s = quarter & 1 ? cr : sr;
        c = quarter & 1 ? sr : cr;
        if (quarter & 2) s = -s;
        if ((quarter + 1) & 2) c = -c;
      }
      cs[t * a.pairs + pair] = c;
      sn[t * a.pairs + pair] = s;
    }
  }
  static size_t bytes(int pairs, int tokens) { return (size_t)pairs * tokens * 8; }
};

// Heads whose rows are whole parts: L lanes a row, 2 N elements a lane, 256 /
// L rows at once. A lane holds both elements of its pairs, so that a rotation is
// within the lane: with pairs half the rotated dimensions apart it has one part
// of each half, otherwise a part of each half of the row. A group walks the heads
// of its tokens, a few rows at once, while the next come by cp.async into a ring in
// shared memory, each lane's own, so that nobody waits for another; the weights
// stay in registers. Arithmetic is packed, two fp32 an instruction.
//
// What bounds it is instruction issue and latency at 16 warps an SM (about 60 % of
// the issue slots), then HBM. 8192x40x128 in bf16 takes 32 us (78 % of the copy
// rate) and 48 backward (78 %). One step ahead in registers instead of the ring:
// 39 and 66. Parts of four elements instead of eight (N): 36 and 54; a layer norm's
// backward pass, with dbeta's sums, has registers for no more than four (eight: 62).
// With four, in three blocks an SM 65 backward, two rows' sums through the shuffles
// together 56. Parts side by side in a lane: 53 instead of 32 for adjacent pairs
// (half of each sector an instruction). Single instructions, partners by shuffles:
// 146 us for 16381x32x128, now 51.
//
// Rows that a lane computes at once; kStages times as many are on their way or computed, 48 KB a block (72 KB for 16-bit
// rows with fp32 gradients, where two stages are 36 us for 34). A fourth stage changes nothing.
template <typename T, typename DT, int N, bool BWD>
struct Ring {
  static constexpr int kRows = !BWD ? 32 / (N * (int)sizeof(T)) : sizeof(T) == 4 || N == 8 ? 1 : 2;
  static constexpr int kX = Part<T, N>::kStride * Part<T, N>::kChunks, kDy = BWD ? Part<DT, N>::kStride * Part<DT, N>::kChunks : 0;
  static constexpr int kStage = 2 * kRows * (kX + kDy), kStages = 3;  // bytes
};

// PLAIN: no layer norm is among the operands.
template <typename T, typename DT, int L, int N, bool BWD, bool INTER, bool PLAIN>
__global__ void __launch_bounds__(kHeadThreads, 2) head_rows(const __grid_constant__ HeadArgs a) {
  using R = Ring<T, DT, N, BWD>;
  constexpr int U = R::kRows;
  constexpr int kGroups = kHeadThreads / L, kStages = R::kStages;
  extern __shared__ __align__(16) unsigned char smem[];
  chained();
  const int which = blockIdx.x >= (unsigned)a.op[0].blocks;
  const HeadOp& o = a.op[which];
  const int block = blockIdx.x - (which ? a.op[0].blocks : 0);
  const Turns turns(smem, a, o.tokens);

  const int li = threadIdx.x % L, group = threadIdx.x / L;
  const int side = 1 << o.shift;  // groups side by side on a token's heads
  const int hh = group & (side - 1), tt = group >> o.shift, step = kGroups >> o.shift;
  const bool on = li * 2 * N < a.D;
  // the lane's quads, its first pair, and which of its pairs turn
  constexpr unsigned kAll = (1u << N) - 1;
  // first and second parts of neighbouring lanes lie side by side: whole sectors
  int d0, d1, pair, pair1;
  unsigned turned = 0;
  if (INTER) {
    d0 = li * N;
    d1 = a.D / 2 + d0;
    pair = (d0 - a.start) / 2;
    pair1 = (d1 - a.start) / 2 - N / 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = (i < N / 2 ? pair : pair1) + i;
      if (on && at >= 0 && at < a.pairs) turned |= 1u << i;
    }
  } else if (li < a.pairs / N) {
    d0 = a.start + N * li;
    d1 = d0 + a.pairs;
    pair = pair1 = N * li;
    turned = kAll;
  } else {  // parts that do not turn
    auto place = [&](int k) { return N * (k < a.start / N ? k : k + 2 * a.pairs / N); };
    d0 = place(li - a.pairs / N);
    d1 = place(li - a.pairs / N + (a.D - 2 * a.pairs) / (2 * N));
    pair = pair1 = 0;
  }
  const long long apart_by = d1 - d0;
  // Whether a lane's factors are whole blocks of four (16384 rows of one head a token: 9.7 us, single ones 11.1).
  const bool by_four = (!INTER || N == 8) && turned == kAll && ((pair | pair1 | a.pairs) & 3) == 0;
  auto weights = [&](const void* w, float none) {
    float x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = on && w ? weight_at(w, a.w_type, d0 + i) : none;
      y[i] = on && w ? weight_at(w, a.w_type, d1 + i) : none;
    }
    return paired<INTER, N>(x, y);
  };
  // wide lanes have no registers for beta, or backward for gamma: it lies behind the table
  constexpr bool kWide = N == 8;
  const Pairs<N> g = weights(BWD && kWide ? nullptr : o.gamma, 1.f), bt = weights(BWD || kWide ? nullptr : o.beta, 0.f);
  float4* const beside = reinterpret_cast<float4*>(smem) + (o.tokens * a.pairs + 1) / 2 + li;
  if (kWide && group == 0 && (BWD || o.beta)) {
    const Pairs<N> e = weights(BWD ? o.gamma : o.beta, BWD ? 1.f : 0.f);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      beside[i * L] = make_float4(e.a[2 * i].x, e.a[2 * i].y, e.a[2 * i + 1].x, e.a[2 * i + 1].y);
      beside[(N / 4 + i) * L] = make_float4(e.b[2 * i].x, e.b[2 * i].y, e.b[2 * i + 1].x, e.b[2 * i + 1].y);
    }
  }
  auto from_beside = [&]() {
    Pairs<N> e;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 x = beside[i * L], y = beside[(N / 4 + i) * L];
      e.a[2 * i] = make_float2(x.x, x.y), e.a[2 * i + 1] = make_float2(x.z, x.w);
      e.b[2 * i] = make_float2(y.x, y.y), e.b[2 * i + 1] = make_float2(y.z, y.w);
    }
    return e;
  };
  Pairs<N> ag{}, ab{};
  const float inv_d = 1.f / (float)a.D;
  const long long x_step = side * o.x_head, y_step = side * o.y_head, dy_step = side * o.dy_head;

  // A lane's rows on their way: kStages times U rows, each lane copies what it takes itself, so that nobody waits for
  // another. A lane without elements holds zeros; groups without a row what was there, which goes nowhere.
  using X = Part<T, N>;
  using DY = Part<DT, N>;
  constexpr int kX = R::kX, kDy = R::kDy, kStage = R::kStage;
  const uint32_t ring = smem_u32(smem + a.ring), x_slot = ring + threadIdx.x * X::kChunk,
                 dy_slot = ring + 2 * U * kX + threadIdx.x * DY::kChunk;
  if (!on)
    for (int i = 0; i < kStages; ++i)
#pragma unroll
      for (int k = 0; k < 2 * U; ++k) {
        X::clear(x_slot + i * kStage + k * kX);
        if (BWD) DY::clear(dy_slot + i * kStage + k * kDy);
      }
  const bool read_x = !BWD || o.norm != IBWD_NORM_NONE;

  // The next rows to load: heads from h0 on of the tokens t0 + tt of a tile.
  struct {
    long long tile;
    int t0, h0;
    bool there;
    const T* x;
    const DT* dy;
  } in{block, 0, 0, false, nullptr, nullptr};
  auto seek_in = [&]() {
    const long long token = in.tile * o.tokens + in.t0 + tt;
    in.there = on && in.tile < o.tiles && in.t0 + tt < o.tokens && token < a.tokens;
    in.x = static_cast<const T*>(o.x) + token * o.x_token + hh * o.x_head + d0;
    if (BWD) in.dy = static_cast<const DT*>(o.dy) + token * o.dy_token + hh * o.dy_head + d0;
  };
  auto load = [&](uint32_t stage) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (in.there && in.h0 + u * side + hh < o.heads) {
        if (read_x) {
          X::copy(x_slot + stage + 2 * u * kX, in.x);
          X::copy(x_slot + stage + (2 * u + 1) * kX, in.x + apart_by);
        }
        if constexpr (BWD) {
          DY::copy(dy_slot + stage + 2 * u * kDy, in.dy);
          DY::copy(dy_slot + stage + (2 * u + 1) * kDy, in.dy + apart_by);
        }
      }
      in.x += x_step;
      if (BWD) in.dy += dy_step;
    }
    cp_async_commit();
    in.h0 += U * side;
    if (in.h0 >= o.heads) {
      in.h0 = 0;
      in.t0 += step;
      if (in.t0 >= o.tokens) {
        in.t0 = 0;
        in.tile += o.blocks;
      }
      seek_in();
    }
  };

  // The rows that are computed, with their token's factors.
  struct {
    long long tile;
    int t0, h0;
    bool there;
    T* y;
  } out{block, 0, 0, false, nullptr};
  float2 c[N / 2], s[N / 2], minus_s[N / 2];
  auto seek_out = [&]() {
    const int t = out.t0 + tt;
    const long long token = out.tile * o.tokens + t;
    out.there = on && t < o.tokens && token < a.tokens;
    out.y = static_cast<T*>(o.y) + token * o.y_token + hh * o.y_head + d0;
    float cc[N], ss[N];
    if (out.there && by_four) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const int at = t * a.pairs + (i < N / 2 ? pair : pair1) + i;
        const float4 x = *reinterpret_cast<const float4*>(turns.cs + at), y = *reinterpret_cast<const float4*>(turns.sn + at);
        cc[i] = x.x, cc[i + 1] = x.y, cc[i + 2] = x.z, cc[i + 3] = x.w;
        ss[i] = y.x, ss[i + 1] = y.y, ss[i + 2] = y.z, ss[i + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool use = out.there && (turned >> i & 1);
        const int at = t * a.pairs + (i < N / 2 ? pair : pair1) + i;
        cc[i] = use ? turns.cs[at] : 1.f;
        ss[i] = use ? turns.sn[at] : 0.f;
      }
    }
    if (BWD)
#pragma unroll
      for (int i = 0; i < N; ++i) ss[i] = -ss[i];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      c[i] = make_float2(cc[2 * i], cc[2 * i + 1]);
      s[i] = make_float2(ss[2 * i], ss[2 * i + 1]);
      minus_s[i] = make_float2(-ss[2 * i], -ss[2 * i + 1]);
    }
  };
  auto store = [&](const Pairs<N>& v, T* y) {
    float e0[N], e1[N];
    apart<INTER, N>(v, e0, e1);
    Part<T, N>::store(y, e0);
    Part<T, N>::store(y + apart_by, e1);
  };
  // y_a = z_a c - z_b s, y_b = z_b c + z_a s, where the pair turns: a rotation may begin or end within the lane
  auto rotate = [&](Pairs<N>& z) {
    if (turned == kAll) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 u = z.a[i], v = z.b[i];
        z.a[i] = fma2(v, minus_s[i], mul2(u, c[i]));
        z.b[i] = fma2(u, s[i], mul2(v, c[i]));
      }
    } else if (turned) {
      auto one = [&](unsigned bit, float& u, float& v, float cs, float sn) {
        if (turned & bit) {
          const float w = u;
          u = fmaf(v, -sn, u * cs);
          v = fmaf(w, sn, v * cs);
        }
      };
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        one(1u << 2 * i, z.a[i].x, z.b[i].x, c[i].x, s[i].x);
        one(2u << 2 * i, z.a[i].y, z.b[i].y, c[i].y, s[i].y);
      }
    }
  };
  auto two = [&](auto part, uint32_t slot, int apart) {
    float e0[N], e1[N];
    part.take(slot);
    part.get(e0);
    part.take(slot + apart);
    part.get(e1);
    return paired<INTER, N>(e0, e1);
  };
  auto elements = [&](uint32_t stage, int u) { return two(X{}, x_slot + stage + 2 * u * kX, kX); };
  const bool layer = !PLAIN && o.norm == IBWD_NORM_LAYER, normed = o.norm != IBWD_NORM_NONE;
  // Rows beyond the heads are computed with what the ring holds, and go nowhere. Forward, the sums of all U rows go
  // through the shuffles together, and the elements are taken apart once more behind them.
  auto forward = [&](uint32_t stage) {
    float rstd[U], minus[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rstd[u] = 1.f;
      minus[u] = 0.f;
    }
    if (normed) {
      if (layer) {
#pragma unroll
        for (int u = 0; u < U; ++u) minus[u] = total(elements(stage, u));
        group_sums<L>(minus);
#pragma unroll
        for (int u = 0; u < U; ++u) minus[u] = on ? minus[u] * -inv_d : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Pairs<N> v = elements(stage, u);
        if (layer) shift(v, minus[u]);
        rstd[u] = product(v, v);
      }
      group_sums<L>(rstd);
#pragma unroll
      for (int u = 0; u < U; ++u) rstd[u] = rsqrtf(fmaf(rstd[u], inv_d, a.eps));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Pairs<N> v = elements(stage, u);
      if (layer) shift(v, minus[u]);
      if (normed) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          v.a[i] = mul2(v.a[i], both(rstd[u]));
          v.b[i] = mul2(v.b[i], both(rstd[u]));
        }
        if (kWide && !o.beta) {
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            v.a[i] = mul2(v.a[i], g.a[i]);
            v.b[i] = mul2(v.b[i], g.b[i]);
          }
        } else {
          const Pairs<N> e = kWide ? from_beside() : bt;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            v.a[i] = fma2(v.a[i], g.a[i], e.a[i]);
            v.b[i] = fma2(v.b[i], g.b[i], e.b[i]);
          }
        }
      }
      rotate(v);
      if (out.there && out.h0 + u * side + hh < o.heads) store(v, out.y);
      out.y += y_step;
    }
  };
  // Backward, row after row, its sums together: with v = x (layer: x - mean),
  // dx = rstd (d - sum(d)/D) - xh (rstd^2 sum(d v)/D).
  auto backward = [&](uint32_t stage) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = out.there && out.h0 + u * side + hh < o.heads;
      Pairs<N> d = two(DY{}, dy_slot + stage + 2 * u * kDy, kDy);
      rotate(d);
      if (normed) {
        Pairs<N> v = elements(stage, u);
        if (layer) {
          float m[1] = {total(v)};
          group_sums<L>(m);
          shift(v, on ? m[0] * -inv_d : 0.f);
        }
        auto times_gamma = [&]() {
          const Pairs<N> w = kWide ? from_beside() : g;
          Pairs<N> e;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            e.a[i] = mul2(d.a[i], w.a[i]);
            e.b[i] = mul2(d.b[i], w.b[i]);
          }
          return e;
        };
        Pairs<N> e = times_gamma();
        float sums[3] = {product(v, v), on ? product(e, v) : 0.f, layer && on ? total(e) : 0.f};
        if (layer) {
          group_sums<L>(sums);
        } else {
          float two[2] = {sums[0], sums[1]};
          group_sums<L>(two);
          sums[0] = two[0];
          sums[1] = two[1];
        }
        const float rstd = rsqrtf(fmaf(sums[0], inv_d, a.eps)), k = rstd * (rstd * sums[1] * -inv_d), less = sums[2] * -inv_d;
        if (kWide) e = times_gamma();  // (again: fewer registers over the sums)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 xa = mul2(v.a[i], both(rstd)), xb = mul2(v.b[i], both(rstd));
          if (live) {
            ag.a[i] = fma2(d.a[i], xa, ag.a[i]);
            ag.b[i] = fma2(d.b[i], xb, ag.b[i]);
            if (layer) {
              ab.a[i] = add2(ab.a[i], d.a[i]);
              ab.b[i] = add2(ab.b[i], d.b[i]);
            }
          }
          if (layer) {
            e.a[i] = add2(e.a[i], both(less));
            e.b[i] = add2(e.b[i], both(less));
          }
          d.a[i] = fma2(xa, both(k), mul2(e.a[i], both(rstd)));
          d.b[i] = fma2(xb, both(k), mul2(e.b[i], both(rstd)));
        }
      }
      if (live) store(d, out.y);
      out.y += y_step;
    }
  };
  // Whether there are more.
  auto compute = [&](uint32_t stage) {
    if constexpr (BWD)
      backward(stage);
    else
      forward(stage);
    out.h0 += U * side;
    if (out.h0 < o.heads) return true;
    out.h0 = 0;
    out.t0 += step;
    if (out.t0 >= o.tokens) {
      out.t0 = 0;
      out.tile += o.blocks;
      if (out.tile >= o.tiles) return false;
      __syncthreads();
      turns.fill(a, out.tile * o.tokens, o.tokens);
      __syncthreads();
    }
    seek_out();
    return true;
  };

  seek_in();
  // (they come while the angles are computed)
  for (int i = 0; i < kStages - 1; ++i) load(i * kStage);
  turns.fill(a, out.tile * o.tokens, o.tokens);
  __syncthreads();
  seek_out();
  uint32_t next = (kStages - 1) * kStage, at = 0;
  while (true) {
    load(next);
    next = next == (kStages - 1) * kStage ? 0 : next + kStage;
    cp_async_wait<kStages - 1>();
    if (!compute(at)) break;
    at = at == (kStages - 1) * kStage ? 0 : at + kStage;
  }

  if (BWD && o.norm != IBWD_NORM_NONE && (o.dgamma || o.dbeta)) {
    // the block's column sums: groups of a warp, then the warps, in a fixed order
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);  // [warps][2][D]
    float x[2][2 * N];
    {
      float p[N], r[N];
      apart<INTER, N>(ag, p, r);
#pragma unroll
      for (int i = 0; i < N; ++i) x[0][i] = p[i], x[0][N + i] = r[i];
      apart<INTER, N>(ab, p, r);
#pragma unroll
      for (int i = 0; i < N; ++i) x[1][i] = p[i], x[1][N + i] = r[i];
    }
#pragma unroll
    for (int i = 0; i < 2 * N; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int w = L; w < 32; w <<= 1) x[k][i] += __shfl_xor_sync(0xffffffffu, x[k][i], w);
        if (on && (threadIdx.x & 31) < L)
          red[((threadIdx.x >> 5) * 2 + k) * a.D + (i < N ? d0 + i : d1 + i - N)] = x[k][i];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += kHeadThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kHeadThreads / 32; ++w) v += red[w * 2 * a.D + i];
      a.part[(long long)blockIdx.x * 2 * a.D + i] = v;
    }
  }
}

// UH rows of a warp, a head every `side`. Every lane loads, places beyond the row or the heads what the last one holds: a
// load under a condition is waited for before the next.
template <typename E, int NE, int UH>
__device__ __forceinline__ void load_any(const void* from, long long token, long long of_head, int h0, int side, int heads, int D,
                                         float (&to)[UH][NE]) {
#pragma unroll
  for (int u = 0; u < UH; ++u) {
    const E* p = static_cast<const E*>(from) + token + min(h0 + u * side, heads - 1) * of_head;
#pragma unroll
    for (int i = 0; i < NE; ++i) to[u][i] = to_f32(p[min((int)(threadIdx.x & 31) + 32 * i, D - 1)]);
  }
}

// Any other heads, up to 32 NE wide: a warp a row, lane l has the elements
// l + 32 i, and a row's rotated pairs meet in shared memory. kRows rows are
// loaded at once, and their sums and their pairs meet at once: bound by the
// latency of these steps. 8192x40x127 in bf16 takes 76 us and 127 backward (33
// and 29 % of the copy rate); row after row in three blocks an SM 140 and 204;
// loads under a condition 150 and 407.
template <int NE, bool BWD>
struct AnyHeads {
  static constexpr int kRows = NE >= 16 ? 1 : NE == 8 ? 2 - BWD : 4, kBlocks = NE >= 16 ? 1 : NE >= 4 ? 2 : 3;
};
template <typename T, int NE, bool BWD>
__global__ void __launch_bounds__(kHeadThreads, AnyHeads<NE, BWD>::kBlocks) head_any(const __grid_constant__ HeadArgs a) {
  constexpr int kWarps = kHeadThreads / 32, UH = AnyHeads<NE, BWD>::kRows;
  extern __shared__ __align__(16) unsigned char smem[];
  chained();
  const int which = blockIdx.x >= (unsigned)a.op[0].blocks;
  const HeadOp& o = a.op[which];
  const int block = blockIdx.x - (which ? a.op[0].blocks : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = reinterpret_cast<float*>(smem) + warp * UH * a.D;
  const Turns turns(smem + (size_t)kWarps * UH * a.D * 4, a, o.tokens);
  const int side = 1 << o.shift;
  const int hh = warp & (side - 1), tt = warp >> o.shift, step = kWarps >> o.shift;
  const float inv_d = 1.f / (float)a.D;
  const bool normed = o.norm != IBWD_NORM_NONE, layer = o.norm == IBWD_NORM_LAYER;
  float ag[BWD ? NE : 1], ab[BWD ? NE : 1], g[NE], bt[BWD ? 1 : NE];
  // of each element: its pair (-1: it does not turn), its partner, and whether it is the first of the two
  int pair[NE], other[NE];
  unsigned first_of = 0;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 32 * i, rel = e - a.start;
    g[i] = e < a.D && o.gamma ? weight_at(o.gamma, a.w_type, e) : 1.f;
    if (!BWD) bt[BWD ? 0 : i] = e < a.D && o.beta ? weight_at(o.beta, a.w_type, e) : 0.f;
    if (BWD) ag[BWD ? i : 0] = ab[BWD ? i : 0] = 0.f;
    pair[i] = -1;
    other[i] = 0;
    if (e < a.D && rel >= 0 && rel < 2 * a.pairs) {
      const bool low = a.interleaved ? !(rel & 1) : rel < a.pairs;
      pair[i] = a.interleaved ? rel >> 1 : low ? rel : rel - a.pairs;
      other[i] = a.start + (a.interleaved ? rel ^ 1 : low ? rel + a.pairs : rel - a.pairs);
      if (low) first_of |= 1u << i;
    }
  }

  for (long long tile = block; tile < o.tiles; tile += o.blocks) {
    const long long first = tile * o.tokens;
    __syncthreads();
    turns.fill(a, first, o.tokens);
    __syncthreads();
    for (int t = tt; t < o.tokens && first + t < a.tokens; t += step) {
      const long long token = first + t;
      float c[NE], s[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        c[i] = pair[i] >= 0 ? turns.cs[t * a.pairs + pair[i]] : 1.f;
        s[i] = pair[i] >= 0 ? turns.sn[t * a.pairs + pair[i]] : 0.f;
        if ((first_of >> i & 1) != (unsigned)BWD) s[i] = -s[i];
      }
      auto rotate = [&](float (&z)[UH][NE]) {
        __syncwarp();
#pragma unroll
        for (int u = 0; u < UH; ++u)
#pragma unroll
          for (int i = 0; i < NE; ++i)
            if (lane + 32 * i < a.D) row[u * a.D + lane + 32 * i] = z[u][i];
        __syncwarp();
#pragma unroll
        for (int u = 0; u < UH; ++u)
#pragma unroll
          for (int i = 0; i < NE; ++i)
            if (pair[i] >= 0) z[u][i] = fmaf(z[u][i], c[i], row[u * a.D + other[i]] * s[i]);
      };
      for (int h0 = hh; h0 < o.heads; h0 += side * UH) {
        float x[UH][NE], dy[UH][NE];
        if (!BWD || normed) load_any<T, NE, UH>(o.x, token * o.x_token, o.x_head, h0, side, o.heads, a.D, x);
        if constexpr (BWD) {
          if (o.dy_f32)
            load_any<float, NE, UH>(o.dy, token * o.dy_token, o.dy_head, h0, side, o.heads, a.D, dy);
          else
            load_any<T, NE, UH>(o.dy, token * o.dy_token, o.dy_head, h0, side, o.heads, a.D, dy);
        }
#pragma unroll
        for (int u = 0; u < UH; ++u)
#pragma unroll
          for (int i = 0; i < NE; ++i)
            if (lane + 32 * i >= a.D) {
              x[u][i] = 0.f;
              if (BWD) dy[u][i] = 0.f;
            }
        float rstd[UH];
        if (normed) {
          if (layer) {
            float m[UH];
#pragma unroll
            for (int u = 0; u < UH; ++u) {
              m[u] = 0.f;
#pragma unroll
              for (int i = 0; i < NE; ++i) m[u] += x[u][i];
            }
            group_sums<32>(m);
#pragma unroll
            for (int u = 0; u < UH; ++u)
#pragma unroll
              for (int i = 0; i < NE; ++i) x[u][i] = lane + 32 * i < a.D ? fmaf(m[u], -inv_d, x[u][i]) : 0.f;
          }
#pragma unroll
          for (int u = 0; u < UH; ++u) {
            rstd[u] = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) rstd[u] = fmaf(x[u][i], x[u][i], rstd[u]);
          }
          group_sums<32>(rstd);
#pragma unroll
          for (int u = 0; u < UH; ++u) {
            rstd[u] = rsqrtf(fmaf(rstd[u], inv_d, a.eps));
#pragma unroll
            for (int i = 0; i < NE; ++i) x[u][i] *= rstd[u];
          }
        }
        if constexpr (!BWD) {
          if (normed)
#pragma unroll
            for (int u = 0; u < UH; ++u)
#pragma unroll
              for (int i = 0; i < NE; ++i) x[u][i] = fmaf(x[u][i], g[i], bt[i]);
          if (a.pairs) rotate(x);
        } else {
          if (a.pairs) rotate(dy);
          if (!normed) {
#pragma unroll
            for (int u = 0; u < UH; ++u)
#pragma unroll
              for (int i = 0; i < NE; ++i) x[u][i] = dy[u][i];
          } else {
            float s1[UH], s2[UH];
#pragma unroll
            for (int u = 0; u < UH; ++u) {
              s1[u] = s2[u] = 0.f;
              const bool live = h0 + u * side < o.heads;
#pragma unroll
              for (int i = 0; i < NE; ++i) {
                if (live) {
                  ag[i] = fmaf(dy[u][i], x[u][i], ag[i]);
                  ab[i] += dy[u][i];
                }
                dy[u][i] *= g[i];
                s1[u] += dy[u][i];
                s2[u] = fmaf(dy[u][i], x[u][i], s2[u]);
              }
            }
            if (layer) group_sums<32>(s1);
            group_sums<32>(s2);
#pragma unroll
            for (int u = 0; u < UH; ++u)
#pragma unroll
              for (int i = 0; i < NE; ++i)
                x[u][i] = rstd[u] * (dy[u][i] - (layer ? s1[u] * inv_d : 0.f) - x[u][i] * (s2[u] * inv_d));
          }
        }
#pragma unroll
        for (int u = 0; u < UH; ++u) {
          const int h = h0 + u * side;
          T* to = static_cast<T*>(o.y) + token * o.y_token + h * o.y_head;
#pragma unroll
          for (int i = 0; i < NE; ++i)
            if (h < o.heads && lane + 32 * i < a.D) to[lane + 32 * i] = from_f32<T>(x[u][i]);
        }
      }
    }
  }
  if constexpr (BWD) {
    if (o.norm != IBWD_NORM_NONE && (o.dgamma || o.dbeta)) {
      __syncthreads();
      float* red = reinterpret_cast<float*>(smem);  // [warps][2][D], over the rows and the table
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = lane + 32 * i;
        if (e < a.D) {
          red[warp * 2 * a.D + e] = ag[i];
          red[warp * 2 * a.D + a.D + e] = ab[i];
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * a.D; i += kHeadThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[w * 2 * a.D + i];
        a.part[(long long)blockIdx.x * 2 * a.D + i] = v;
      }
    }
  }
}

// How a launch splits its tokens: tiles of tokens, whose heads go to the
// block's `groups` rows at once.  Few groups side by side on a token's heads
// give a group several heads for one set of the rotation's factors; more of
// them where that would leave SMs without a tile. All blocks are resident and
// walk their tiles, shared out between the operands by cost.
inline void plan_heads(HeadArgs* a, int groups, int per_sm, int side_by, bool backward) {
  const int resident = per_sm * a->num_sms, budget = backward && resident > kHeadBlocks ? kHeadBlocks : resident;
  // what a token costs an operand: its heads, and its angles, as much as about eight heads
  const int angles = a->pairs ? 8 : 1;
  for (int w = 0; w < 2; ++w) {
    HeadOp& o = a->op[w];
    o.shift = 0;
    o.tokens = 1;
    o.blocks = 0;
    o.tiles = 0;
    if (!o.heads || !a->tokens) continue;
    while ((1 << (o.shift + 1)) <= groups && (side_by << (o.shift + 1)) <= o.heads) ++o.shift;
    auto tiles = [&](int tokens) { return (a->tokens + tokens - 1) / tokens; };
    while ((1 << o.shift) < groups && (1 << o.shift) < o.heads && tiles(groups >> o.shift) < a->num_sms) ++o.shift;
    o.tokens = groups >> o.shift;
    // several tokens a group while there are tiles enough and the table of angles stays at 16 KB
    const int rows = (o.heads + (1 << o.shift) - 1) >> o.shift;
    for (int m = rows; m < 8 && tiles(2 * o.tokens) >= 4 * a->num_sms && 2 * o.tokens * a->pairs <= kHeadAngles; m *= 2) o.tokens *= 2;
    o.tiles = tiles(o.tokens);
    o.blocks = (int)(o.tiles < budget ? o.tiles : budget);
  }
  HeadOp &q = a->op[0], &k = a->op[1];
  if (q.tiles + k.tiles <= budget || !q.tiles || !k.tiles) return;
  // The split whose longest blocks take least: whole tiles, so that one operand's blocks all have as many, or the other's.
  const long long costs[2] = {q.tokens * (q.heads + angles), k.tokens * (k.heads + angles)};
  long long least = LLONG_MAX;
  auto turns = [](long long n, long long by) { return (n + by - 1) / by; };
  for (int w = 0; w < 2; ++w) {
    const long long n = a->op[w].tiles, m = a->op[1 - w].tiles;
    const long long ideal = (n * costs[w] + m * costs[1 - w]) / (budget * costs[w]);
    for (long long r = ideal > 1 ? ideal : 1; r <= ideal + 2; ++r) {
      const long long mine = turns(n, r), rest = budget - mine < m ? budget - mine : m;
      if (rest < 1) continue;
      const long long t = turns(m, rest) * costs[1 - w], most = r * costs[w] > t ? r * costs[w] : t;
      if (most >= least) continue;
      least = most;
      a->op[w].blocks = (int)mine;
      a->op[1 - w].blocks = (int)rest;
    }
  }
}

// Whether every row of an operand is whole parts of n elements.
inline bool heads_aligned(const void* p, long long token, long long head, int size, int n) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (n * size < 16 ? n * size : 16) == 0 && token % n == 0 && head % n == 0);
}

// [blocks][2][D] column sums of the kernels above to dgamma and dbeta.
cudaError_t join_heads(const HeadArgs& a, cudaStream_t st);

template <typename T, bool BWD>
cudaError_t launch_heads_of(HeadArgs a, cudaStream_t st) {
  auto whole = [&](int n) {
    bool is = a.D % (2 * n) == 0 && a.D <= 256 && (a.interleaved ? a.start % 2 == 0 : a.start % n == 0 && a.pairs % n == 0);
    for (const HeadOp& o : a.op)
      if (o.heads)
        is = is && heads_aligned(o.x, o.x_token, o.x_head, sizeof(T), n) && heads_aligned(o.y, o.y_token, o.y_head, sizeof(T), n) &&
             (!BWD || heads_aligned(o.dy, o.dy_token, o.dy_head, o.dy_f32 ? 4 : (int)sizeof(T), n));
    return is;
  };
  // Wide lanes have 16 elements' weights to load first: 320 rows take 3.4 us, with them 3.9; 5120 4.6 and 4.7; 16384
  // 13.0 and 11.2; 327680 36 and 32.
  const bool rows = whole(4), plain = a.op[0].norm != IBWD_NORM_LAYER && a.op[1].norm != IBWD_NORM_LAYER,
             wide = (!BWD || plain) && sizeof(T) == 2 && a.tokens * (a.op[0].heads + a.op[1].heads) >= 8192 && whole(8);
  int lanes = wide ? 4 : 8;
  while (lanes * (wide ? 16 : 8) < a.D) lanes *= 2;
  if (!rows) lanes = 32;
  struct {
    int rows, blocks;
  } any{AnyHeads<16, BWD>::kRows, AnyHeads<16, BWD>::kBlocks};
  if (a.D <= 256) any = {AnyHeads<8, BWD>::kRows, AnyHeads<8, BWD>::kBlocks};
  if (a.D <= 128) any = {AnyHeads<4, BWD>::kRows, AnyHeads<4, BWD>::kBlocks};
  if (a.D <= 64) any = {AnyHeads<2, BWD>::kRows, AnyHeads<2, BWD>::kBlocks};  // (and of one)
  plan_heads(&a, kHeadThreads / lanes, rows ? 2 : any.blocks, wide ? 8 : 16, BWD);
  const unsigned grid = a.op[0].blocks + a.op[1].blocks;
  if (grid) {
    const int tokens = a.op[0].tokens > a.op[1].tokens ? a.op[0].tokens : a.op[1].tokens;
    const size_t table = (Turns::bytes(a.pairs, tokens) + 15) / 16 * 16 + (wide ? lanes * 64 : 0), sums = (size_t)(kHeadThreads / 32) * 2 * a.D * 4;
    const size_t used = rows ? table : table + (size_t)(kHeadThreads / 32) * any.rows * a.D * 4;
    const size_t base = ((BWD && sums > used ? sums : used) + 15) / 16 * 16;  // at most 32 KB
    a.ring = (int)base;
    auto launch = [&](const HeadArgs& b, unsigned blocks, bool f32) {
      auto go = [&](auto kern) { return launch_ex(kern, blocks, kHeadThreads, base, st, true, b); };
      auto by_lanes = [&](auto dt) {
        using DT = decltype(dt);
        auto ringed = [&](auto lanes_of, auto n, auto inter) {
          constexpr int L = decltype(lanes_of)::value, N = decltype(n)::value;
          constexpr bool INTER = decltype(inter)::value;
          static std::atomic<size_t> done[64];
          const auto kern = head_rows<T, DT, L, N, BWD, INTER, BWD && N == 8>;
          constexpr size_t ring = (size_t)Ring<T, DT, N, BWD>::kStages * Ring<T, DT, N, BWD>::kStage;
          if (base > kHeadFront) return cudaErrorInvalidValue;  // (never)
          // The limit is that of the largest front, whatever this launch has: another thread's may have more.
          const cudaError_t e = raise_smem(reinterpret_cast<const void*>(kern), kHeadFront + ring, done);
          return e != cudaSuccess ? e : launch_ex(kern, blocks, kHeadThreads, base + ring, st, true, b);
        };
        auto by_inter = [&](auto lanes_of, auto n) {
          return a.interleaved ? ringed(lanes_of, n, std::true_type{}) : ringed(lanes_of, n, std::false_type{});
        };
        if constexpr (sizeof(T) == 2)
          if (wide) {
            constexpr std::integral_constant<int, 8> n{};
            if (lanes == 4) return by_inter(std::integral_constant<int, 4>{}, n);
            if (lanes == 8) return by_inter(std::integral_constant<int, 8>{}, n);
            return by_inter(std::integral_constant<int, 16>{}, n);
          }
        constexpr std::integral_constant<int, 4> n{};
        if (lanes == 8) return by_inter(std::integral_constant<int, 8>{}, n);
        if (lanes == 16) return by_inter(std::integral_constant<int, 16>{}, n);
        return by_inter(std::integral_constant<int, 32>{}, n);
      };
      if (!rows) {
        if (a.D <= 32) return go(head_any<T, 1, BWD>);
        if (a.D <= 64) return go(head_any<T, 2, BWD>);
        if (a.D <= 128) return go(head_any<T, 4, BWD>);
        return a.D <= 256 ? go(head_any<T, 8, BWD>) : go(head_any<T, 16, BWD>);
      }
      if constexpr (BWD)
        if (f32) return by_lanes(float{});
      return by_lanes(T{});
    };
    cudaError_t e;
    if (rows && BWD && a.op[0].heads && a.op[1].heads && a.op[0].dy_f32 != a.op[1].dy_f32) {
      // gradients of two types: a launch each, its sums where one launch would have them
      HeadArgs q = a, k = a;
      q.op[1].blocks = k.op[0].blocks = 0;
      k.part = a.part ? a.part + (long long)a.op[0].blocks * 2 * a.D : nullptr;
      e = launch(q, a.op[0].blocks, a.op[0].dy_f32);
      if (e == cudaSuccess) e = launch(k, a.op[1].blocks, a.op[1].dy_f32);
    } else {
      e = launch(a, grid, a.op[a.op[0].heads ? 0 : 1].dy_f32);
    }
    if (e != cudaSuccess) return e;
  }
  if (!BWD) return cudaSuccess;
  return join_heads(a, st);
}

}  // namespace ibwd
