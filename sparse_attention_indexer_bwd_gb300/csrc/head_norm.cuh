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

namespace ibwd {

constexpr int kHeadThreads = 256;

__device__ __forceinline__ float weight_at(const void* w, int type, int i) {
  if (type == IBWD_F32) return static_cast<const float*>(w)[i];
  if (type == IBWD_BF16) return to_f32(static_cast<const __nv_bfloat16*>(w)[i]);
  return to_f32(static_cast<const __half*>(w)[i]);
}

// Four elements side by side, as they lie in memory.
template <typename T>
struct Quad {
  uint2 w;
  // Two quads where `live`, into the registers that they have: loads that are selected afterwards would be waited for at once.
  __device__ static void load(Quad (&q)[2], const T* p0, const T* p1, bool live) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t@p ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%4];\n\t"
                 "@p ld.global.L1::no_allocate.v2.u32 {%2,%3}, [%5];\n\t}"
                 : "+r"(q[0].w.x), "+r"(q[0].w.y), "+r"(q[1].w.x), "+r"(q[1].w.y)
                 : "l"(p0), "l"(p1), "r"((int)live));
  }
  __device__ void zero() { w = make_uint2(0, 0); }
  __device__ void get(float (&v)[4]) const {
    const float2 a = unpack2(w.x, T{}), b = unpack2(w.y, T{});
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
  __device__ static void store(T* p, const float (&v)[4]) {
    const uint32_t a = pack2_of(make_float2(v[0], v[1]), T{}), b = pack2_of(make_float2(v[2], v[3]), T{});
    asm volatile("st.global.L1::no_allocate.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(a), "r"(b) : "memory");
  }
};
template <>
struct Quad<float> {
  uint4 w;
  __device__ static void load(Quad (&q)[2], const float* p0, const float* p1, bool live) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %10, 0;\n\t@p ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%8];\n\t"
                 "@p ld.global.L1::no_allocate.v4.u32 {%4,%5,%6,%7}, [%9];\n\t}"
                 : "+r"(q[0].w.x), "+r"(q[0].w.y), "+r"(q[0].w.z), "+r"(q[0].w.w), "+r"(q[1].w.x), "+r"(q[1].w.y),
                   "+r"(q[1].w.z), "+r"(q[1].w.w)
                 : "l"(p0), "l"(p1), "r"((int)live));
  }
  __device__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&v)[4]) const { unpack(w, v, 0.f); }
  __device__ static void store(float* p, const float (&v)[4]) {
    st_stream(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
  }
};

// A lane's eight elements of a row: partners a_i and b_i of four pairs, packed
// by twos (two fp32 an instruction).
struct Eight {
  float2 a[2], b[2];
};
// INTER: quads (a0 b0 a1 b1) and (a2 b2 a3 b3); otherwise (a0 .. a3) and (b0 .. b3).
template <bool INTER>
__device__ __forceinline__ Eight paired(const float (&x)[4], const float (&y)[4]) {
  Eight e;
  if (INTER) {
    e.a[0] = make_float2(x[0], x[2]), e.b[0] = make_float2(x[1], x[3]);
    e.a[1] = make_float2(y[0], y[2]), e.b[1] = make_float2(y[1], y[3]);
  } else {
    e.a[0] = make_float2(x[0], x[1]), e.a[1] = make_float2(x[2], x[3]);
    e.b[0] = make_float2(y[0], y[1]), e.b[1] = make_float2(y[2], y[3]);
  }
  return e;
}
template <bool INTER>
__device__ __forceinline__ void apart(const Eight& e, float (&x)[4], float (&y)[4]) {
  if (INTER) {
    x[0] = e.a[0].x, x[1] = e.b[0].x, x[2] = e.a[0].y, x[3] = e.b[0].y;
    y[0] = e.a[1].x, y[1] = e.b[1].x, y[2] = e.a[1].y, y[3] = e.b[1].y;
  } else {
    x[0] = e.a[0].x, x[1] = e.a[0].y, x[2] = e.a[1].x, x[3] = e.a[1].y;
    y[0] = e.b[0].x, y[1] = e.b[0].y, y[2] = e.b[1].x, y[3] = e.b[1].y;
  }
}
__device__ __forceinline__ float total(const Eight& v) {
  const float2 t = add2(add2(v.a[0], v.a[1]), add2(v.b[0], v.b[1]));
  return t.x + t.y;
}
__device__ __forceinline__ float product(const Eight& v, const Eight& w) {
  const float2 t = fma2(v.b[1], w.b[1], fma2(v.b[0], w.b[0], fma2(v.a[1], w.a[1], mul2(v.a[0], w.a[0]))));
  return t.x + t.y;
}
__device__ __forceinline__ void shift(Eight& v, float by) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
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
    freq = (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0);
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

// Heads whose rows are whole quads: L lanes a row, eight elements a lane, 256 /
// L rows at once. A lane holds both elements of its pairs, so that a rotation is
// within the lane: with pairs half the rotated dimensions apart it has one quad
// of each half (two 8-byte loads of a 16-bit type), otherwise two quads side by
// side. A group walks the heads of its tokens, U rows at once while the next U
// are on their way, kept as they lie in memory; the weights stay in registers.
// Arithmetic is packed, two fp32 an instruction: with single instructions, and
// partners fetched by shuffles, 16381x32x128 took 146 us, bound by issue at
// 16 warps an SM.
template <typename T, typename DT, int L, bool BWD, bool INTER>
__global__ void __launch_bounds__(kHeadThreads, 2) head_rows(const __grid_constant__ HeadArgs a) {
  constexpr int U = !BWD ? 4 : sizeof(T) == 4 ? 1 : 2;
  constexpr int kGroups = kHeadThreads / L;
  extern __shared__ __align__(16) unsigned char smem[];
  chained();
  const int which = blockIdx.x >= (unsigned)a.op[0].blocks;
  const HeadOp& o = a.op[which];
  const int block = blockIdx.x - (which ? a.op[0].blocks : 0);
  const Turns turns(smem, a, o.tokens);

  const int li = threadIdx.x % L, group = threadIdx.x / L;
  const int side = 1 << o.shift;  // groups side by side on a token's heads
  const int hh = group & (side - 1), tt = group >> o.shift, step = kGroups >> o.shift;
  const bool on = li * 8 < a.D;
  // the lane's quads, its first pair, and which of its four pairs turn
  int d0 = li * 8, d1 = li * 8 + 4, pair = 0;
  unsigned turned = 0;
  if (INTER) {
    const int rel = d0 - a.start;
    pair = rel / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (on && rel + 2 * i >= 0 && rel + 2 * i < 2 * a.pairs) turned |= 1u << i;
  } else if (li < a.pairs / 4) {
    d0 = a.start + 4 * li;
    d1 = d0 + a.pairs;
    pair = 4 * li;
    turned = 15u;
  } else {  // quads that do not turn, by twos
    auto place = [&](int k) { return 4 * (k < a.start / 4 ? k : k + a.pairs / 2); };
    d0 = place(2 * (li - a.pairs / 4));
    d1 = place(2 * (li - a.pairs / 4) + 1);
  }
  const long long apart_by = d1 - d0;
  auto weights = [&](const void* w, float none) {
    float x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = on && w ? weight_at(w, a.w_type, d0 + i) : none;
      y[i] = on && w ? weight_at(w, a.w_type, d1 + i) : none;
    }
    return paired<INTER>(x, y);
  };
  const Eight g = weights(o.gamma, 1.f), bt = weights(BWD ? nullptr : o.beta, 0.f);
  Eight ag{}, ab{};
  const float inv_d = 1.f / (float)a.D;
  const long long x_step = side * o.x_head, y_step = side * o.y_head, dy_step = side * o.dy_head;

  // U rows of a lane. A lane without elements holds zeros; groups without a row what they had, which goes nowhere.
  struct Rows {
    Quad<T> x[U][2];
    Quad<DT> dy[BWD ? U : 1][2];
  };
  Rows rows[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        rows[i].x[u][k].zero();
        if (BWD) rows[i].dy[BWD ? u : 0][k].zero();
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
  auto load = [&](Rows& r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = in.there && in.h0 + u * side + hh < o.heads;
      if (read_x) Quad<T>::load(r.x[u], in.x, in.x + apart_by, live);
      if constexpr (BWD) Quad<DT>::load(r.dy[u], in.dy, in.dy + apart_by, live);
      in.x += x_step;
      if (BWD) in.dy += dy_step;
    }
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
  float2 c[2], s[2], minus_s[2];
  auto seek_out = [&]() {
    const int t = out.t0 + tt;
    const long long token = out.tile * o.tokens + t;
    out.there = on && t < o.tokens && token < a.tokens;
    out.y = static_cast<T*>(o.y) + token * o.y_token + hh * o.y_head + d0;
    float cc[4], ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool use = out.there && (turned >> i & 1);
      cc[i] = use ? turns.cs[t * a.pairs + pair + i] : 1.f;
      ss[i] = use ? turns.sn[t * a.pairs + pair + i] : 0.f;
      if (BWD) ss[i] = -ss[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = make_float2(cc[2 * i], cc[2 * i + 1]);
      s[i] = make_float2(ss[2 * i], ss[2 * i + 1]);
      minus_s[i] = make_float2(-ss[2 * i], -ss[2 * i + 1]);
    }
  };
  auto store = [&](const Eight& v, T* y) {
    float e0[4], e1[4];
    apart<INTER>(v, e0, e1);
    Quad<T>::store(y, e0);
    Quad<T>::store(y + apart_by, e1);
  };
  // y_a = z_a c - z_b s, y_b = z_b c + z_a s, where the pair turns: a rotation may begin or end within the lane
  auto rotate = [&](Eight& z) {
    if (turned == 15u) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
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
      one(1u, z.a[0].x, z.b[0].x, c[0].x, s[0].x);
      one(2u, z.a[0].y, z.b[0].y, c[0].y, s[0].y);
      one(4u, z.a[1].x, z.b[1].x, c[1].x, s[1].x);
      one(8u, z.a[1].y, z.b[1].y, c[1].y, s[1].y);
    }
  };
  auto elements = [&](const Quad<T> (&x)[2]) {
    float e0[4], e1[4];
    x[0].get(e0);
    x[1].get(e1);
    return paired<INTER>(e0, e1);
  };
  const bool layer = o.norm == IBWD_NORM_LAYER, normed = o.norm != IBWD_NORM_NONE;
  // Rows beyond the heads are computed with what the registers hold, and go nowhere. Forward, the sums of all U rows go
  // through the shuffles together, and the elements are taken apart once more behind them (row after row: 42 us for 40).
  auto forward = [&](const Rows& r) {
    float rstd[U], minus[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rstd[u] = 1.f;
      minus[u] = 0.f;
    }
    if (normed) {
      if (layer) {
#pragma unroll
        for (int u = 0; u < U; ++u) minus[u] = total(elements(r.x[u]));
        group_sums<L>(minus);
#pragma unroll
        for (int u = 0; u < U; ++u) minus[u] = on ? minus[u] * -inv_d : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Eight v = elements(r.x[u]);
        if (layer) shift(v, minus[u]);
        rstd[u] = product(v, v);
      }
      group_sums<L>(rstd);
#pragma unroll
      for (int u = 0; u < U; ++u) rstd[u] = rsqrtf(fmaf(rstd[u], inv_d, a.eps));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Eight v = elements(r.x[u]);
      if (layer) shift(v, minus[u]);
      if (normed) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          v.a[i] = fma2(mul2(v.a[i], both(rstd[u])), g.a[i], bt.a[i]);
          v.b[i] = fma2(mul2(v.b[i], both(rstd[u])), g.b[i], bt.b[i]);
        }
      }
      rotate(v);
      if (out.there && out.h0 + u * side + hh < o.heads) store(v, out.y);
      out.y += y_step;
    }
  };
  // Backward, row after row (two at once spill: 82 us for 66 at 8192x40x128 bf16), its sums together: with v = x (layer: x - mean),
  // dx = rstd (d - sum(d)/D) - xh (rstd^2 sum(d v)/D).
  auto backward = [&](const Rows& r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = out.there && out.h0 + u * side + hh < o.heads;
      float e0[4], e1[4];
      r.dy[u][0].get(e0);
      r.dy[u][1].get(e1);
      Eight d = paired<INTER>(e0, e1);
      rotate(d);
      if (normed) {
        Eight v = elements(r.x[u]);
        if (layer) {
          float m[1] = {total(v)};
          group_sums<L>(m);
          shift(v, on ? m[0] * -inv_d : 0.f);
        }
        Eight e;  // d gamma
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e.a[i] = mul2(d.a[i], g.a[i]);
          e.b[i] = mul2(d.b[i], g.b[i]);
        }
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
#pragma unroll
        for (int i = 0; i < 2; ++i) {
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
  auto compute = [&](const Rows& r) {
    if constexpr (BWD)
      backward(r);
    else
      forward(r);
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
  load(rows[0]);  // (they come while the angles are computed)
  turns.fill(a, out.tile * o.tokens, o.tokens);
  __syncthreads();
  seek_out();
  while (true) {
    load(rows[1]);
    if (!compute(rows[0])) break;
    load(rows[0]);
    if (!compute(rows[1])) break;
  }

  if (BWD && o.norm != IBWD_NORM_NONE && (o.dgamma || o.dbeta)) {
    // the block's column sums: groups of a warp, then the warps, in a fixed order
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);  // [warps][2][D]
    float x[2][8];
    {
      float p[4], r[4];
      apart<INTER>(ag, p, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[0][i] = p[i], x[0][4 + i] = r[i];
      apart<INTER>(ab, p, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[1][i] = p[i], x[1][4 + i] = r[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int w = L; w < 32; w <<= 1) x[k][i] += __shfl_xor_sync(0xffffffffu, x[k][i], w);
        if (on && (threadIdx.x & 31) < L)
          red[((threadIdx.x >> 5) * 2 + k) * a.D + (i < 4 ? d0 + i : d1 + i - 4)] = x[k][i];
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
// l + 32 i, and a row's rotated pairs meet in shared memory. UH rows are loaded at once.
template <typename T, int NE, bool BWD>
__global__ void __launch_bounds__(kHeadThreads, NE == 4 ? 3 : 1) head_any(const __grid_constant__ HeadArgs a) {
  constexpr int kWarps = kHeadThreads / 32, UH = NE > 4 ? 1 : BWD ? 2 : 4;
  extern __shared__ __align__(16) unsigned char smem[];
  chained();
  const int which = blockIdx.x >= (unsigned)a.op[0].blocks;
  const HeadOp& o = a.op[which];
  const int block = blockIdx.x - (which ? a.op[0].blocks : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = reinterpret_cast<float*>(smem) + warp * a.D;
  const Turns turns(smem + (size_t)kWarps * a.D * 4, a, o.tokens);
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
      auto rotate = [&](float (&z)[NE]) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (lane + 32 * i < a.D) row[lane + 32 * i] = z[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (pair[i] >= 0) z[i] = fmaf(z[i], c[i], row[other[i]] * s[i]);
      };
      for (int h0 = hh; h0 < o.heads; h0 += side * UH) {
        float x[UH][NE], dy[BWD ? UH : 1][NE];
#pragma unroll
        for (int u = 0; u < UH; ++u) {
          const int h = h0 + u * side;
          const T* px = static_cast<const T*>(o.x) + token * o.x_token + h * o.x_head + lane;
          const long long pd = token * o.dy_token + h * o.dy_head + lane;
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            const bool on = h < o.heads && lane + 32 * i < a.D;
            x[u][i] = 0.f;
            if (on && (!BWD || normed)) x[u][i] = to_f32(px[32 * i]);
            if (BWD) {
              dy[BWD ? u : 0][i] = 0.f;
              if (on)
                dy[BWD ? u : 0][i] = o.dy_f32 ? static_cast<const float*>(o.dy)[pd + 32 * i] : to_f32(static_cast<const T*>(o.dy)[pd + 32 * i]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < UH; ++u) {
          const int h = h0 + u * side;
          if (h >= o.heads) break;  // (alike in the warp)
          float(&v)[NE] = x[u];
          float rstd = 1.f;
          if (normed) {
            if (layer) {
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
            rstd = rsqrtf(fmaf(warp_sum(q), inv_d, a.eps));
#pragma unroll
            for (int i = 0; i < NE; ++i) v[i] *= rstd;
          }
          if constexpr (!BWD) {
            if (normed)
#pragma unroll
              for (int i = 0; i < NE; ++i) v[i] = fmaf(v[i], g[i], bt[i]);
            if (a.pairs) rotate(v);
          } else {
            float(&d)[NE] = dy[u];
            if (a.pairs) rotate(d);
            if (!normed) {
#pragma unroll
              for (int i = 0; i < NE; ++i) v[i] = d[i];
            } else {
              float s1 = 0.f, s2 = 0.f;
#pragma unroll
              for (int i = 0; i < NE; ++i) {
                if (lane + 32 * i < a.D) {
                  ag[i] = fmaf(d[i], v[i], ag[i]);
                  ab[i] += d[i];
                  d[i] *= g[i];
                  s1 += d[i];
                  s2 = fmaf(d[i], v[i], s2);
                }
              }
              s1 = layer ? warp_sum(s1) * inv_d : 0.f;
              s2 = warp_sum(s2) * inv_d;
#pragma unroll
              for (int i = 0; i < NE; ++i) v[i] = rstd * (d[i] - s1 - v[i] * s2);
            }
          }
#pragma unroll
          for (int i = 0; i < NE; ++i)
            if (lane + 32 * i < a.D)
              static_cast<T*>(o.y)[token * o.y_token + h * o.y_head + lane + 32 * i] = from_f32<T>(v[i]);
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
inline void plan_heads(HeadArgs* a, int groups, int per_sm, bool backward) {
  const int resident = per_sm * a->num_sms, budget = backward && resident > kHeadBlocks ? kHeadBlocks : resident;
  // what a token costs an operand: its heads, and its angles, as much as about eight heads
  const int angles = a->pairs ? 8 : 1, first = a->op[0].heads + angles, both = first + a->op[1].heads + angles;
  for (int w = 0; w < 2; ++w) {
    HeadOp& o = a->op[w];
    o.shift = 0;
    o.tokens = 1;
    o.blocks = 0;
    o.tiles = 0;
    if (!o.heads || !a->tokens) continue;
    while ((1 << (o.shift + 1)) <= groups && (16 << (o.shift + 1)) <= o.heads) ++o.shift;
    auto tiles = [&](int tokens) { return (a->tokens + tokens - 1) / tokens; };
    while ((1 << o.shift) < groups && (1 << o.shift) < o.heads && tiles(groups >> o.shift) < a->num_sms) ++o.shift;
    o.tokens = groups >> o.shift;
    // several tokens a group while there are tiles enough and the table of angles stays at 16 KB
    const int rows = (o.heads + (1 << o.shift) - 1) >> o.shift;
    for (int m = rows; m < 8 && tiles(2 * o.tokens) >= 4 * a->num_sms && 2 * o.tokens * a->pairs <= 2048; m *= 2) o.tokens *= 2;
    o.tiles = tiles(o.tokens);
    int share = budget;
    if (a->op[0].heads && a->op[1].heads) {
      share = (int)((long long)budget * first / both);
      share = share < 1 ? 1 : share > budget - 1 ? budget - 1 : share;
      if (w) share = budget - share;
    }
    o.blocks = (int)(o.tiles < share ? o.tiles : share);
  }
}

// Whether every row of an operand is whole quads.
inline bool heads_aligned(const void* p, long long token, long long head, int size) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && token % 4 == 0 && head % 4 == 0);
}

// [blocks][2][D] column sums of the kernels above to dgamma and dbeta.
cudaError_t join_heads(const HeadArgs& a, cudaStream_t st);

template <typename T, bool BWD>
cudaError_t launch_heads_of(HeadArgs a, cudaStream_t st) {
  bool rows = a.D % 8 == 0 && a.D <= 256 && (a.interleaved ? a.start % 2 == 0 : a.start % 4 == 0 && a.pairs % 4 == 0);
  for (const HeadOp& o : a.op)
    if (o.heads)
      rows = rows && heads_aligned(o.x, o.x_token, o.x_head, sizeof(T)) && heads_aligned(o.y, o.y_token, o.y_head, sizeof(T)) &&
             (!BWD || heads_aligned(o.dy, o.dy_token, o.dy_head, o.dy_f32 ? 4 : (int)sizeof(T)));
  int lanes = 8;
  while (lanes * 8 < a.D) lanes *= 2;
  if (!rows) lanes = 32;
  plan_heads(&a, kHeadThreads / lanes, rows ? 2 : a.D <= 128 ? 3 : 1, BWD);
  const unsigned grid = a.op[0].blocks + a.op[1].blocks;
  if (grid) {
    const int tokens = a.op[0].tokens > a.op[1].tokens ? a.op[0].tokens : a.op[1].tokens;
    const size_t table = Turns::bytes(a.pairs, tokens), sums = (size_t)(kHeadThreads / 32) * 2 * a.D * 4;
    // at most 36 KB, which a launch has without asking: 512 wide rows, and 2048 pairs' factors
    const size_t used = rows ? table : table + (size_t)(kHeadThreads / 32) * a.D * 4;
    const size_t bytes = BWD && sums > used ? sums : used;
    auto launch = [&](const HeadArgs& b, unsigned blocks, bool f32) {
      auto go = [&](auto kern) { return launch_ex(kern, blocks, kHeadThreads, bytes, st, true, b); };
      auto by_lanes = [&](auto dt) {
        using DT = decltype(dt);
        if (lanes == 8) return a.interleaved ? go(head_rows<T, DT, 8, BWD, true>) : go(head_rows<T, DT, 8, BWD, false>);
        if (lanes == 16) return a.interleaved ? go(head_rows<T, DT, 16, BWD, true>) : go(head_rows<T, DT, 16, BWD, false>);
        return a.interleaved ? go(head_rows<T, DT, 32, BWD, true>) : go(head_rows<T, DT, 32, BWD, false>);
      };
      if (!rows) return a.D <= 128 ? go(head_any<T, 4, BWD>) : go(head_any<T, 16, BWD>);
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
