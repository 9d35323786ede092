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

namespace ibwd {

constexpr int kHeadThreads = 256;

__device__ __forceinline__ float weight_at(const void* w, int type, int i) {
  if (type == IBWD_F32) return static_cast<const float*>(w)[i];
  if (type == IBWD_BF16) return to_f32(static_cast<const __nv_bfloat16*>(w)[i]);
  return to_f32(static_cast<const __half*>(w)[i]);
}

// Eight elements of a row, 16-byte aligned.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) { unpack(ld_stream(p), v, __nv_bfloat16{}); }
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) { unpack(ld_stream(p), v, __half{}); }
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  float a[4], b[4];
  unpack(ld_stream(p), a, 0.f);
  unpack(ld_stream(p + 4), b, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2_of(make_float2(v[2 * i], v[2 * i + 1]), T{});
  st_stream(p, make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  st_stream(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
  st_stream(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
}

// Sum over a group of L lanes, in every one of them.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The rotation of a tile's tokens in shared memory: [tokens][pairs] cosines,
// then sines, filled by the whole block; every head of a token takes them from
// there, so that their 40 instructions a pair are spent once a token and
// operand (per head they would be three times the norm's).
struct Turns {
  unsigned long long* freq;  // [pairs] fraction of a turn
  int* axis;
  float* cs;
  float* sn;

  __device__ Turns(unsigned char* smem, const HeadArgs& a, int tokens) {
    freq = reinterpret_cast<unsigned long long*>(smem);
    cs = reinterpret_cast<float*>(freq + a.pairs);
    sn = cs + tokens * a.pairs;
    axis = reinterpret_cast<int*>(sn + tokens * a.pairs);
  }
  __device__ void init(const HeadArgs& a) const {
    for (int i = threadIdx.x; i < a.pairs; i += kHeadThreads) {
      const double f = a.freq64 ? static_cast<const double*>(a.freq)[i] : (double)static_cast<const float*>(a.freq)[i];
      const double turns = f * 0.15915494309189533577;  // 1 / 2 pi
      freq[i] = (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0);
      axis[i] = a.axis_of ? a.axis_of[i] : 0;
    }
  }
  __device__ void fill(const HeadArgs& a, long long first, int tokens) const {
    const long long left = a.tokens - first;
    for (int idx = threadIdx.x; idx < tokens * a.pairs; idx += kHeadThreads) {
      const int t = idx / a.pairs, i = idx - t * a.pairs;
      float s = 0.f, c = 1.f;
      // an axis that does not exist turns nothing
      if (t < left && (unsigned)axis[i] < (unsigned)a.axes) {
        const long long at = axis[i] * a.axis_stride + first + t;
        const long long pos = a.positions64 ? static_cast<const long long*>(a.positions)[at]
                                            : (long long)static_cast<const int*>(a.positions)[at];
        const int turn = (int)((freq[i] * (unsigned long long)pos) >> 32);  // 2^-32 turns
        const int quarter = (int)(((unsigned)turn + 0x20000000u) >> 30);
        const float r = (float)(int)((unsigned)turn - ((unsigned)quarter << 30)) * 0x1p-31f;  // half turns
        float sr, cr;
        sincospif(r, &sr, &cr);
        s = quarter & 1 ? cr : sr;
        c = quarter & 1 ? sr : cr;
        if (quarter & 2) s = -s;
        if ((quarter + 1) & 2) c = -c;
      }
      cs[idx] = c;
      sn[idx] = s;
    }
  }
  static size_t bytes(int pairs, int tokens) { return (size_t)pairs * 12 + (size_t)pairs * tokens * 8; }
};

// Heads whose rows are 16-byte blocks: L lanes a row, eight elements a lane,
// 256 / L rows at once. A group walks the heads of its tokens with U rows in
// flight; the rotation's factors and the weights stay in registers. A lane's
// partners in the other half of the rotated dimensions come by shuffles.
template <typename T, int L, bool BWD>
__global__ void __launch_bounds__(kHeadThreads) head_rows(const __grid_constant__ HeadArgs a) {
  constexpr int U = BWD ? 2 : 4;
  constexpr int kGroups = kHeadThreads / L;
  extern __shared__ __align__(16) unsigned char smem[];
  const int which = blockIdx.x >= (unsigned)a.op[0].blocks;
  const HeadOp& o = a.op[which];
  const int block = blockIdx.x - (which ? a.op[0].blocks : 0);
  const Turns turns(smem, a, o.tokens);
  turns.init(a);

  const int li = threadIdx.x % L, group = threadIdx.x / L;
  const int side = 1 << o.shift;  // groups side by side on a token's heads
  const int hh = group & (side - 1), tt = group >> o.shift, step = kGroups >> o.shift;
  const int dim = li * 8;
  const bool on = dim < a.D;
  const int turned = 2 * a.pairs, rel = dim - a.start;
  const bool mine = on && rel >= 0 && rel < turned;
  // lane of the other half's eight dimensions
  const int partner = mine && !a.interleaved ? (threadIdx.x & 31) + (rel < a.pairs ? a.pairs / 8 : -(a.pairs / 8))
                                             : (threadIdx.x & 31);
  float g[8], b[8], ag[8], ab[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] = on && o.gamma ? weight_at(o.gamma, a.w_type, dim + i) : 1.f;
    b[i] = !BWD && on && o.beta ? weight_at(o.beta, a.w_type, dim + i) : 0.f;
    ag[i] = ab[i] = 0.f;
  }
  const float inv_d = 1.f / (float)a.D;

  for (long long tile = block; tile < o.tiles; tile += o.blocks) {
    const long long first = tile * o.tokens;
    __syncthreads();  // freq, or the tile before
    turns.fill(a, first, o.tokens);
    __syncthreads();
    for (int t0 = 0; t0 < o.tokens; t0 += step) {
      const int t = t0 + tt;
      const bool there = first + t < a.tokens && t < o.tokens;
      // y_e = z_e c_e + z_partner(e) s_e
      float c[8], s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
      }
      if (mine && there) {
        const float *pc = turns.cs + t * a.pairs, *ps = turns.sn + t * a.pairs;
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (rel + 2 * i < turned) {
              const int p = rel / 2 + i;
              c[2 * i] = c[2 * i + 1] = pc[p];
              s[2 * i] = BWD ? ps[p] : -ps[p];
              s[2 * i + 1] = -s[2 * i];
            }
        } else {
          const bool low = rel < a.pairs;
          const int p = low ? rel : rel - a.pairs;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            c[i] = pc[p + i];
            s[i] = low != BWD ? -ps[p + i] : ps[p + i];
          }
        }
      }
      auto rotate = [&](float (&z)[8]) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = z[2 * i], v = z[2 * i + 1];
            if (mine && rel + 2 * i < turned) {
              z[2 * i] = fmaf(u, c[2 * i], v * s[2 * i]);
              z[2 * i + 1] = fmaf(v, c[2 * i], u * s[2 * i + 1]);
            }
          }
        } else if (a.pairs) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float v = __shfl_sync(0xffffffffu, z[i], partner);
            z[i] = mine ? fmaf(z[i], c[i], v * s[i]) : z[i];
          }
        }
      };
      const long long token = first + t;
      for (int h0 = 0; h0 < o.heads; h0 += U * side) {
        float x[U][8], dy[BWD ? U : 1][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * side + hh;
          const bool live = there && on && h < o.heads;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[u][i] = 0.f;
            if (BWD) dy[BWD ? u : 0][i] = 0.f;
          }
          if (live) {
            if (!BWD || o.norm != IBWD_NORM_NONE) load8(static_cast<const T*>(o.x) + token * o.x_token + h * o.x_head + dim, x[u]);
            if (BWD) {
              const long long at = token * o.dy_token + h * o.dy_head + dim;
              if (o.dy_f32)
                load8(static_cast<const float*>(o.dy) + at, dy[BWD ? u : 0]);
              else
                load8(static_cast<const T*>(o.dy) + at, dy[BWD ? u : 0]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * side + hh;
          if (h0 + u * side >= o.heads) break;  // (alike in all groups)
          float(&v)[8] = x[u];
          float rstd = 1.f;
          if (o.norm != IBWD_NORM_NONE) {
            if (o.norm == IBWD_NORM_LAYER) {
              float m = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) m += v[i];
              m = group_sum<L>(m) * inv_d;
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = on ? v[i] - m : 0.f;
            }
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) q = fmaf(v[i], v[i], q);
            rstd = 1.f / sqrtf(group_sum<L>(q) * inv_d + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= rstd;
          }
          if (!BWD) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], g[i], b[i]);
            rotate(v);
          } else {
            float(&d)[8] = dy[BWD ? u : 0];
            rotate(d);
            if (o.norm == IBWD_NORM_NONE) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = d[i];
            } else {
              float s1 = 0.f, s2 = 0.f;
              const bool live = there && h < o.heads;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (live) {
                  ag[i] = fmaf(d[i], v[i], ag[i]);
                  ab[i] += d[i];
                }
                d[i] *= g[i];
                s1 += d[i];
                s2 = fmaf(d[i], v[i], s2);
              }
              s1 = o.norm == IBWD_NORM_LAYER ? group_sum<L>(on ? s1 : 0.f) * inv_d : 0.f;
              s2 = group_sum<L>(on ? s2 : 0.f) * inv_d;
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = rstd * (d[i] - s1 - v[i] * s2);
            }
          }
          if (there && on && h < o.heads) store8(static_cast<T*>(o.y) + token * o.y_token + h * o.y_head + dim, v);
        }
      }
    }
  }

  if (BWD) griddep_launch_dependents();
  if (BWD && o.norm != IBWD_NORM_NONE && (o.dgamma || o.dbeta)) {
    // the block's column sums: groups of a warp, then the warps, in a fixed order
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);  // [warps][2][D]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int w = L; w < 32; w <<= 1) {
        ag[i] += __shfl_xor_sync(0xffffffffu, ag[i], w);
        ab[i] += __shfl_xor_sync(0xffffffffu, ab[i], w);
      }
      if (on && (threadIdx.x & 31) < L) {
        float* r = red + (threadIdx.x >> 5) * 2 * a.D + dim + i;
        r[0] = ag[i];
        r[a.D] = ab[i];
      }
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

// Any other heads, up to 32 NE wide: a warp a row, lane l has the elements
// l + 32 i, and a row's rotated pairs meet in shared memory.
template <typename T, int NE, bool BWD>
__global__ void __launch_bounds__(kHeadThreads) head_any(const __grid_constant__ HeadArgs a) {
  constexpr int kWarps = kHeadThreads / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  const int which = blockIdx.x >= (unsigned)a.op[0].blocks;
  const HeadOp& o = a.op[which];
  const int block = blockIdx.x - (which ? a.op[0].blocks : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = reinterpret_cast<float*>(smem) + warp * a.D;
  const Turns turns(smem + (size_t)kWarps * a.D * 4, a, o.tokens);
  turns.init(a);
  const int side = 1 << o.shift;
  const int hh = warp & (side - 1), tt = warp >> o.shift, step = kWarps >> o.shift;
  const float inv_d = 1.f / (float)a.D;
  float ag[BWD ? NE : 1], ab[BWD ? NE : 1];
#pragma unroll
  for (int i = 0; i < (BWD ? NE : 1); ++i) ag[i] = ab[i] = 0.f;

  for (long long tile = block; tile < o.tiles; tile += o.blocks) {
    const long long first = tile * o.tokens;
    __syncthreads();
    turns.fill(a, first, o.tokens);
    __syncthreads();
    for (int t = tt; t < o.tokens && first + t < a.tokens; t += step) {
      const long long token = first + t;
      // z turned by the token's angles, backward by minus them
      auto rotate = [&](float (&z)[NE]) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (lane + 32 * i < a.D) row[lane + 32 * i] = z[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int rel = lane + 32 * i - a.start;
          if (lane + 32 * i < a.D && rel >= 0 && rel < 2 * a.pairs) {
            const bool low = a.interleaved ? !(rel & 1) : rel < a.pairs;
            const int p = a.interleaved ? rel >> 1 : low ? rel : rel - a.pairs;
            const float other = row[a.start + (a.interleaved ? rel ^ 1 : low ? rel + a.pairs : p)];
            const float c = turns.cs[t * a.pairs + p], s = turns.sn[t * a.pairs + p];
            z[i] = fmaf(z[i], c, other * (low != BWD ? -s : s));
          }
        }
      };
      for (int h = hh; h < o.heads; h += side) {
        float v[NE], d[BWD ? NE : 1];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int e = lane + 32 * i;
          v[i] = 0.f;
          if (e < a.D && (!BWD || o.norm != IBWD_NORM_NONE))
            v[i] = to_f32(static_cast<const T*>(o.x)[token * o.x_token + h * o.x_head + e]);
          if (BWD) {
            const long long at = token * o.dy_token + h * o.dy_head + e;
            d[BWD ? i : 0] = e >= a.D ? 0.f
                             : o.dy_f32 ? static_cast<const float*>(o.dy)[at]
                                        : to_f32(static_cast<const T*>(o.dy)[at]);
          }
        }
        float rstd = 1.f;
        if (o.norm != IBWD_NORM_NONE) {
          if (o.norm == IBWD_NORM_LAYER) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) m += v[i];
            m = warp_sum(m) * inv_d;
#pragma unroll
            for (int i = 0; i < NE; ++i) v[i] = lane + 32 * i < a.D ? v[i] - m : 0.f;
          }
          float q = 0.f;
#pragma unroll
          for (int i = 0; i < NE; ++i) q = fmaf(v[i], v[i], q);
          rstd = 1.f / sqrtf(warp_sum(q) * inv_d + a.eps);
#pragma unroll
          for (int i = 0; i < NE; ++i) v[i] *= rstd;
        }
        if constexpr (!BWD) {
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            const int e = lane + 32 * i;
            if (e < a.D && o.norm != IBWD_NORM_NONE)
              v[i] = fmaf(v[i], o.gamma ? weight_at(o.gamma, a.w_type, e) : 1.f,
                          o.beta ? weight_at(o.beta, a.w_type, e) : 0.f);
          }
          if (a.pairs) rotate(v);
        } else {
          if (a.pairs) rotate(d);
          if (o.norm == IBWD_NORM_NONE) {
#pragma unroll
            for (int i = 0; i < NE; ++i) v[i] = d[i];
          } else {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
              const int e = lane + 32 * i;
              if (e < a.D) {
                ag[i] = fmaf(d[i], v[i], ag[i]);
                ab[i] += d[i];
                if (o.gamma) d[i] *= weight_at(o.gamma, a.w_type, e);
              }
              s1 += d[i];
              s2 = fmaf(d[i], v[i], s2);
            }
            s1 = o.norm == IBWD_NORM_LAYER ? warp_sum(s1) * inv_d : 0.f;
            s2 = warp_sum(s2) * inv_d;
#pragma unroll
            for (int i = 0; i < NE; ++i) v[i] = rstd * (d[i] - s1 - v[i] * s2);
          }
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int e = lane + 32 * i;
          if (e < a.D) static_cast<T*>(o.y)[token * o.y_token + h * o.y_head + e] = from_f32<T>(v[i]);
        }
      }
    }
  }
  if constexpr (BWD) {
    griddep_launch_dependents();
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
// them where that would leave SMs without a tile.  Blocks of a backward pass
// are as many as the workspace holds sums of, shared out by heads.
inline void plan_heads(HeadArgs* a, int groups, bool backward) {
  const int budget = backward ? kHeadBlocks : 1 << 30;
  const int all = a->op[0].heads + a->op[1].heads;
  for (int w = 0; w < 2; ++w) {
    HeadOp& o = a->op[w];
    o.shift = 0;
    o.tokens = 1;
    o.blocks = 0;
    o.tiles = 0;
    if (!o.heads || !a->tokens) continue;
    while ((1 << (o.shift + 1)) <= groups && (4 << (o.shift + 1)) <= o.heads) ++o.shift;
    auto tiles = [&](int tokens) { return (a->tokens + tokens - 1) / tokens; };
    while ((1 << o.shift) < groups && (1 << o.shift) < o.heads && tiles(groups >> o.shift) < a->num_sms) ++o.shift;
    o.tokens = groups >> o.shift;
    // several tokens a group while there are tiles enough and the table of angles stays at 16 KB
    const int rows = (o.heads + (1 << o.shift) - 1) >> o.shift;
    for (int m = rows; m < 8 && tiles(2 * o.tokens) >= 4 * a->num_sms && 2 * o.tokens * a->pairs <= 2048; m *= 2) o.tokens *= 2;
    o.tiles = tiles(o.tokens);
    int share = budget;
    if (backward && a->op[0].heads && a->op[1].heads) {
      share = (int)((long long)kHeadBlocks * a->op[0].heads / all);
      share = share < 1 ? 1 : share > kHeadBlocks - 1 ? kHeadBlocks - 1 : share;
      if (w) share = kHeadBlocks - share;
    }
    o.blocks = (int)(o.tiles < share ? o.tiles : share);
  }
}

// Whether every row of an operand is whole 16-byte blocks.
inline bool heads_aligned(const void* p, long long token, long long head, int size) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && token * size % 16 == 0 && head * size % 16 == 0);
}

// [blocks][2][D] column sums of the kernels above to dgamma and dbeta; `behind`: launched right behind them.
cudaError_t join_heads(const HeadArgs& a, bool behind, cudaStream_t st);

template <typename T, bool BWD>
cudaError_t launch_heads_of(HeadArgs a, cudaStream_t st) {
  bool rows = a.D % 8 == 0 && a.D <= 256 && a.start % 8 == 0 && (a.interleaved || a.pairs % 8 == 0);
  for (const HeadOp& o : a.op)
    if (o.heads)
      rows = rows && heads_aligned(o.x, o.x_token, o.x_head, sizeof(T)) && heads_aligned(o.y, o.y_token, o.y_head, sizeof(T)) &&
             (!BWD || heads_aligned(o.dy, o.dy_token, o.dy_head, o.dy_f32 ? 4 : (int)sizeof(T)));
  int lanes = 4;
  while (lanes * 8 < a.D) lanes *= 2;
  if (!rows) lanes = 32;
  plan_heads(&a, kHeadThreads / lanes, BWD);
  const unsigned grid = a.op[0].blocks + a.op[1].blocks;
  if (grid) {
    const int tokens = a.op[0].tokens > a.op[1].tokens ? a.op[0].tokens : a.op[1].tokens;
    const size_t table = Turns::bytes(a.pairs, tokens), sums = (size_t)(kHeadThreads / 32) * 2 * a.D * 4;
    // at most 36 KB, which a launch has without asking: 512 wide rows, and 2048 pairs' factors
    const size_t used = rows ? table : table + (size_t)(kHeadThreads / 32) * a.D * 4;
    const size_t bytes = BWD && sums > used ? sums : used;
    cudaError_t e;
    auto go = [&](auto kern) { return launch_ex(kern, grid, kHeadThreads, bytes, st, false, a); };
    if (!rows)
      e = a.D <= 128 ? go(head_any<T, 4, BWD>) : go(head_any<T, 16, BWD>);
    else if (lanes == 4)
      e = go(head_rows<T, 4, BWD>);
    else if (lanes == 8)
      e = go(head_rows<T, 8, BWD>);
    else if (lanes == 16)
      e = go(head_rows<T, 16, BWD>);
    else
      e = go(head_rows<T, 32, BWD>);
    if (e != cudaSuccess) return e;
  }
  if (!BWD) return cudaSuccess;
  return join_heads(a, grid != 0, st);
}

}  // namespace ibwd
