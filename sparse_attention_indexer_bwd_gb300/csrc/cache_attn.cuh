// Attention over the paged 8-bit cache, for one or a few query tokens a
// sequence:
//   s_t = scale q . k_t,  p = softmax(s),  out = sum p_t v_t,  lse = log sum exp(s_t).
//
// Bound by the codes' bytes, 2 D a token and KV head, as long as a KV head's
// queries are few: each code is read once for all rows (query tokens x heads of
// the group) of a KV head, 16 or 32 rows a tile.
//
// The work is a list of tiles of 64 positions (sequences, KV heads, row tiles,
// positions, in that order), cut into equal runs, one a block, wherever that
// falls: lengths are read on the device, so ragged batches and single long
// sequences fill the SMs alike. A block joins its four warps at the end of an
// item (a row tile of a KV head of a sequence); an item that lies in several
// blocks is joined by a second kernel, launched programmatically behind the
// first, in the order of the blocks.
//
// A warp works alone on 16 positions of a tile: cp.async brings their codes to
// its own ring of stages, mma.sync takes them as fp16 (each code, e4m3 or
// int8, is exact there). The contraction over D runs in an order that gives a
// lane 16 contiguous codes of a key, the same for the query; values are
// transposed by ldmatrix in pairs of bytes. tcgen05 would want 128 rows of
// queries and the codes written to shared memory once more in fp16: with 4 to
// 32 rows its tiles would be mostly padding.
//
// Two running maxima a row: m of the logits (base 2) for the sum l, and M of
// logit + log2(scale of the value's block), which is what the outputs' unit
// follows, so that a weight has 11 bits relative to the largest contribution
// whatever the blocks' scales are. Weights are kept in units of 2^-15, at most
// 2^15 in fp16: they lose bits only below 2^-29 of the largest and vanish below 2^-39.
#pragma once
#include "cache.h"
#include "elem.cuh"
#include "indexer_cache.h"
#include "kcommon.cuh"
#include "ptx.cuh"
#include "train.h"

#include <climits>
#include <type_traits>

namespace ibwd {

constexpr int kTile = 64;          // positions of a block's step
constexpr int kAttnThreads = 128;  // four warps, 16 positions each
constexpr int kAttnGrid = 456;     // blocks at most, which is what the workspace holds
constexpr float kUnit = 15.f;      // log2 of the largest weight in fp16

// What a block leaves for the join: the item that it ends without having begun it.
struct JoinRecord {
  int valid, first;  // the first block of the item
  int token, row;    // its first query token, the tile's first row
  int rows, head;    // rows of the KV head's queries, the KV head
  int pad[2];
};

// Floats of one partial result's row: outputs, m, l, M.
constexpr int part_row(int D) { return D + 4; }

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
// Bytes of u (int8 + 128) at SEL's places as a pair of fp16: 1024 + byte, less 1152.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t int8_pair(uint32_t u) {
  const uint32_t h = __byte_perm(u, 0x64646464u, SEL), m = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&m));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Four codes as two pairs of fp16: (0, 1) and (2, 3).
template <bool INT8>
__device__ __forceinline__ void adjacent(uint32_t w, uint32_t& a, uint32_t& b) {
  if (INT8) {
    w ^= 0x80808080u;
    a = int8_pair<0x4140>(w);
    b = int8_pair<0x4342>(w);
  } else {
    a = e4m3_pair(w & 0xFFFFu);
    b = e4m3_pair(w >> 16);
  }
}
// The same: (0, 2) and (1, 3).
template <bool INT8>
__device__ __forceinline__ void alternate(uint32_t w, uint32_t& a, uint32_t& b) {
  if (INT8) {
    w ^= 0x80808080u;
    a = int8_pair<0x4240>(w);
    b = int8_pair<0x4341>(w);
  } else {
    w = __byte_perm(w, 0, 0x3120);
    a = e4m3_pair(w & 0xFFFFu);
    b = e4m3_pair(w >> 16);
  }
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half_pair(float a, float b) { return pack2_of(make_float2(a, b), __half{}); }
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
// What a maximum is subtracted as: -inf (nothing yet) as 0.
__device__ __forceinline__ float basis(float m) { return m == -INFINITY ? 0.f : m; }

// Where 16 bytes of a stage's row lie: ldmatrix takes eight rows at once, and a
// lane's quarter of a key two, without a bank conflict.
template <int D>
__device__ __forceinline__ int stage_at(int row, int chunk) {
  if (D == 64) return row * 64 + ((chunk ^ (row >> 1 & 3)) << 4);
  return row * D + ((chunk ^ (row & 7)) << 4);
}

// The items in their order, and the tiles of the current one.
template <int ROWS, bool SEL>
struct Cursor {
  int b;        // sequence; with SEL the query token
  int head, rt;
  int tile, tiles;
  int row_tiles, rows;  // row tiles and rows of a KV head
  int token;            // first query token
  int len;              // positions held; with SEL places of the list
  int seen;             // positions that the first query token sees
  int seq;

  __device__ void enter(const CacheAttnArgs& a) {
    const CacheSeqs& s = a.seqs;
    if (SEL) {
      token = b;
      seq = b;
      if (s.cu) {  // the last sequence that begins at or before the token
        int lo = 0, hi = s.batch;
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32, at = lo + (int)(threadIdx.x & 31) * step;
          const unsigned below = __ballot_sync(0xffffffffu, at < hi && (at == lo || s.begin(at) <= b));
          lo += (__popc(below) - 1) * step;
          hi = min(hi, lo + step);
        }
        seq = lo;
      }
      const long long at = (long long)s.lens[seq] - s.begin(seq + 1) + b;
      seen = (int)max(0ll, min(at + 1, (long long)s.length(seq)));
      rows = a.group;
      len = a.kept;
    } else {
      seq = b;
      token = s.begin(b);
      const int n = max(0, s.begin(b + 1) - token);
      len = n ? s.length(b) : 0;
      seen = n ? (int)max(-(1ll << 30), min((long long)s.lens[b] - n + 1, 1ll << 30)) : 0;
      rows = (int)min((long long)n * a.group, 1ll << 30);
    }
    row_tiles = (rows + ROWS - 1) / ROWS;
    tiles = max(1, (len + kTile - 1) / kTile);
  }
  // Moves on by one tile; whether that ends the item.
  __device__ bool step(const CacheAttnArgs& a) {
    if (++tile < tiles) return false;
    tile = 0;
    if (++rt < row_tiles) return true;
    rt = 0;
    if (++head < a.heads) return true;
    head = 0;
    const int end = SEL ? (int)a.seqs.tokens : a.seqs.batch;
    do {
      if (++b >= end) return true;
      enter(a);
    } while (!rows);
    return true;
  }
};

// Tiles of sequence b.
template <int ROWS>
__device__ __forceinline__ long long tiles_of(const CacheAttnArgs& a, int b) {
  const CacheSeqs& s = a.seqs;
  const long long n = s.begin(b + 1) - s.begin(b);
  if (n <= 0) return 0;
  return (n * a.group + ROWS - 1) / ROWS * a.heads * max(1, (s.length(b) + kTile - 1) / kTile);
}

template <int D, int MT, bool INT8, bool SEL, int STAGES, int BLOCKS>
__global__ void __launch_bounds__(kAttnThreads, BLOCKS) attn_kernel(const __grid_constant__ CacheAttnArgs a, bool vec) {
  constexpr int ROWS = 16 * MT, kRowChunks = D / 16, kBytes = 16 * D;
  constexpr int kStage = 2 * kBytes + 160;  // keys, values, 16 scales of each, a mask
  constexpr int kLane = D / 64;             // 16-byte chunks of a key that a lane takes
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long scan[5];
  __shared__ int found_b;
  __shared__ long long found_rest;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane & 3;
  const CacheSeqs& s = a.seqs;

  // ------------------------------------------------- this block's run of tiles
  using Place = Cursor<ROWS, SEL>;
  Place c;
  long long total, t0, t1;
  long long blocks;  // that have tiles: at least one each, since the join takes a part of each
  c.head = c.rt = c.tile = 0;
  if (SEL) {
    const int tokens = s.cu ? s.begin(s.batch) : (int)s.tokens;
    const long long each = (long long)((a.group + ROWS - 1) / ROWS) * a.heads * ((a.kept + kTile - 1) / kTile);
    total = each * tokens;
    blocks = min((long long)gridDim.x, total);
    t0 = blockIdx.x < blocks ? total * blockIdx.x / blocks : 0;
    t1 = blockIdx.x < blocks ? total * (blockIdx.x + 1) / blocks : 0;
    c.b = (int)(t0 / each);
    found_rest = t0 - c.b * each;  // (alike in all threads)
  } else {
    const int per = (s.batch + kAttnThreads - 1) / kAttnThreads;
    const int b0 = min((int)threadIdx.x * per, s.batch), b1 = min(b0 + per, s.batch);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += tiles_of<ROWS>(a, b);
    long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kAttnThreads / 32; ++w) {
      if (w < warp) upto += scan[w];
      total += scan[w];
    }
    blocks = min((long long)gridDim.x, total);
    t0 = blockIdx.x < blocks ? total * blockIdx.x / blocks : 0;
    t1 = blockIdx.x < blocks ? total * (blockIdx.x + 1) / blocks : 0;
    if (t0 >= upto - sum && t0 < upto) {
      long long rest = t0 - (upto - sum);
      int b = b0;
      for (; b < b1; ++b) {
        const long long n = tiles_of<ROWS>(a, b);
        if (rest < n) break;
        rest -= n;
      }
      found_b = b;
      found_rest = rest;
    }
    __syncthreads();
    c.b = found_b;
  }
  JoinRecord* record = static_cast<JoinRecord*>(a.work) + blockIdx.x;
  float* parts = reinterpret_cast<float*>(static_cast<JoinRecord*>(a.work) + kAttnGrid);
  if (t0 >= t1) {
    if (threadIdx.x == 0) record->valid = 0;
    griddep_launch_dependents();
    return;
  }
  if (SEL) __syncthreads();
  long long rest = found_rest;
  c.enter(a);
  {
    const long long per_head = (long long)c.row_tiles * c.tiles;
    c.head = (int)(rest / per_head);
    rest -= c.head * per_head;
    c.rt = (int)(rest / c.tiles);
    c.tile = (int)(rest - (long long)c.rt * c.tiles);
  }
  if (threadIdx.x == 0) {
    const long long begin = t0 - c.tile;
    JoinRecord r{};
    if (c.tile > 0 && begin + c.tiles <= t1) {
      r.valid = 1;
      r.first = (int)(((begin + 1) * blocks - 1) / total);
      r.token = c.token;
      r.row = c.rt * ROWS;
      r.rows = c.rows;
      r.head = c.head;
    }
    *record = r;
  }

  // ------------------------------------------------------------------- loads
  unsigned char* ring = smem + warp * (STAGES * kStage);
  float* stats = reinterpret_cast<float*>(smem + 4 * STAGES * kStage);  // [4][ROWS][3]
  float* join = stats + 4 * ROWS * 3 + 16;                              // [2][16][D + 4]
  const int P = 1 << s.page_log;
  Place l = c;
  int left = (int)min(t1 - t0, (long long)INT_MAX);  // tiles to be loaded
  // what the next load takes: this lane's position (dense: the first one) and its page
  int at = 0, page = -1, listed = -1;
  auto look_up = [&]() {
    at = l.tile * kTile + warp * 16;
    if (SEL) {
      const int place = at + (lane & 15);
      listed = left > 0 && place < a.kept ? a.select[(long long)l.token * a.kept + place] : -1;
    } else {
      page = left > 0 && at < l.len ? s.page_at(l.seq, at) : -1;
    }
  };
  auto look_up_page = [&]() {
    if (SEL) {
      at = listed;
      page = listed >= 0 && listed < l.seen ? s.page_at(l.seq, listed) : -1;
    }
  };
  auto load = [&](int stage) {
    if (left > 0) {
      unsigned char* to = ring + stage * kStage;
      const uint32_t to32 = smem_u32(to);
      unsigned mask;
      long long row = 0;
      const long long block = (long long)page * a.heads + l.head;
      if (SEL) {
        mask = __ballot_sync(0xffffffffu, page >= 0) & 0xFFFFu;
        if (page >= 0) row = (block << s.page_log) + (at & (P - 1));
      } else {
        mask = page < 0 ? 0u : l.len - at >= 16 ? 0xFFFFu : (1u << (l.len - at)) - 1u;
        if (page >= 0) row = (block << s.page_log) + (at & (P - 1));
      }
      if (mask) {
#pragma unroll
        for (int i = 0; i < kRowChunks / 2; ++i) {
          const int idx = i * 32 + lane, r = idx / kRowChunks, ch = idx % kRowChunks;
          const long long src = ((SEL ? __shfl_sync(0xffffffffu, row, r) : row + r) * D) + ch * 16;
          const uint32_t bytes = mask >> r & 1 ? 16u : 0u;
          const uint32_t dst = to32 + stage_at<D>(r, ch);
          cp_async16(dst, static_cast<const uint8_t*>(a.k) + (bytes ? src : 0), bytes);
          cp_async16(dst + kBytes, static_cast<const uint8_t*>(a.v) + (bytes ? src : 0), bytes);
        }
        if (lane < 16) {
          const bool on = mask >> lane & 1;
          cp_async4(to32 + 2 * kBytes + 4 * lane, a.k_scale + (on ? block : 0), on ? 4u : 0u);
          cp_async4(to32 + 2 * kBytes + 64 + 4 * lane, a.v_scale + (on ? block : 0), on ? 4u : 0u);
        }
      }
      if (lane == 0) *reinterpret_cast<unsigned*>(to + 2 * kBytes + 128) = mask;
      if (--left > 0) l.step(a);
    }
    cp_async_commit();
  };
  look_up();
  look_up_page();
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    load(i);
    look_up();
    look_up_page();
  }

  // ------------------------------------------------------------------- items
  uint32_t q[MT][D / 16][4];
  float qs[MT][2], m[MT][2], big[MT][2], sum[MT][2];
  int lim[MT][2], lim_min = 0;
  float o[MT][D / 8][4];
  bool begun = c.tile == 0;  // the segment at hand holds its item's first tile

  auto enter_item = [&]() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = c.rt * ROWS + mt * 16 + hf * 8 + (lane >> 2);
        const bool on = r < c.rows;
        const int i = r / a.group;
        lim[mt][hf] = SEL ? 0 : on ? c.seen + i : -1;
        const long long from = on ? (long long)(c.token + i) * a.q_token + (long long)(c.head * a.group + r - i * a.group) * a.q_head : 0;
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + from;
        float amax = 0.f;
        uint4 raw[kLane][2];
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
          const int ch = D == 64 ? j : (k >> 1) * 8 + 2 * j + (k & 1);
          raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
          if (on) {
            if (vec) {
              raw[k][0] = *reinterpret_cast<const uint4*>(p + ch * 16);
              raw[k][1] = *reinterpret_cast<const uint4*>(p + ch * 16 + 8);
            } else {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = (uint32_t)p[ch * 16 + 2 * e] | (uint32_t)p[ch * 16 + 2 * e + 1] << 16;
              raw[k][0] = make_uint4(w[0], w[1], w[2], w[3]);
              raw[k][1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          const uint32_t w[8] = {raw[k][0].x, raw[k][0].y, raw[k][0].z, raw[k][0].w,
                                 raw[k][1].x, raw[k][1].y, raw[k][1].z, raw[k][1].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = a.type == IBWD_BF16 ? unpack2(w[e], __nv_bfloat16{}) : unpack2(w[e], __half{});
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        amax = quad_max(amax);
        // the row in units of 2^e with its largest entry in [1, 2), and 2^-e; an infinity leaves its finite neighbours finite
        const int e = amax == INFINITY ? 113 : min((int)(__float_as_uint(amax) >> 23) - 127, 126);
        const float down = amax == 0.f || e < -126 ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23);
        qs[mt][hf] = (amax == 0.f || e < -126 ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23)) * a.scale_log2;
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
          const uint32_t w[8] = {raw[k][0].x, raw[k][0].y, raw[k][0].z, raw[k][0].w,
                                 raw[k][1].x, raw[k][1].y, raw[k][1].z, raw[k][1].w};
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float2 f = a.type == IBWD_BF16 ? unpack2(w[g], __nv_bfloat16{}) : unpack2(w[g], __half{});
            // word g / 2 of the chunk is a step of 16 dimensions: its first pair, then its second
            q[mt][k * 4 + g / 2][(g & 1) * 2 + hf] = half_pair(f.x * down, f.y * down);
          }
        }
        m[mt][hf] = big[mt][hf] = -INFINITY;
        sum[mt][hf] = 0.f;
      }
    lim_min = c.seen + c.rt * ROWS / a.group;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
  };

  // Joins the warps' results of the segment: to `out` where it is the whole item, else to the block's parts.
  auto leave_item = [&](bool whole) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        sum[mt][hf] = quad_sum(sum[mt][hf]);
        if (j == 0) {
          float* p = stats + (warp * ROWS + mt * 16 + hf * 8 + (lane >> 2)) * 3;
          p[0] = m[mt][hf];
          p[1] = sum[mt][hf];
          p[2] = big[mt][hf];
        }
      }
    __syncthreads();
    float tm[MT][2], tl[MT][2], tb[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float* p = stats + (mt * 16 + hf * 8 + (lane >> 2)) * 3;
        float mm = -INFINITY, bb = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mm = fmaxf(mm, p[w * ROWS * 3]);
          bb = fmaxf(bb, p[w * ROWS * 3 + 2]);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) ll += p[w * ROWS * 3 + 1] * ex2(p[w * ROWS * 3] - basis(mm));
        tm[mt][hf] = mm;
        tl[mt][hf] = ll;
        tb[mt][hf] = bb;
        const float f = ex2(big[mt][hf] - basis(bb));
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[mt][i][2 * hf] *= f;
          o[mt][i][2 * hf + 1] *= f;
        }
      }
    // (of each pair of n-tiles a lane has four dimensions side by side)
    auto put = [&](float* to, int mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float4*>(to + (hf * 8 + (lane >> 2)) * (D + 4) + i * 16 + 4 * j) =
              make_float4(o[mt][2 * i][2 * hf], o[mt][2 * i + 1][2 * hf], o[mt][2 * i][2 * hf + 1], o[mt][2 * i + 1][2 * hf + 1]);
    };
    auto add = [&](const float* from, int mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(from + (hf * 8 + (lane >> 2)) * (D + 4) + i * 16 + 4 * j);
          o[mt][2 * i][2 * hf] += v.x;
          o[mt][2 * i + 1][2 * hf] += v.y;
          o[mt][2 * i][2 * hf + 1] += v.z;
          o[mt][2 * i + 1][2 * hf + 1] += v.w;
        }
    };
    constexpr int kHalf = 16 * (D + 4);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt) __syncthreads();
      if (warp >= 2) put(join + (warp - 2) * kHalf, mt);
      __syncthreads();
      if (warp < 2) add(join + warp * kHalf, mt);
      __syncthreads();
      if (warp == 1) put(join, mt);
      __syncthreads();
      if (warp == 0) add(join, mt);
    }
    if (warp) return;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = mt * 16 + hf * 8 + (lane >> 2), R = c.rt * ROWS + r;
        if (R >= c.rows) continue;
        if (whole) {
          const int i = R / a.group;
          const long long row = (long long)(c.token + i) * a.heads * a.group + c.head * a.group + R - i * a.group;
          const float l2 = tl[mt][hf];
          const float f = l2 == 0.f ? 0.f : ex2(tb[mt][hf] - kUnit - basis(tm[mt][hf])) / l2;
          uint16_t* to = static_cast<uint16_t*>(a.out) + row * D + 4 * j;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            const float2 x = make_float2(o[mt][2 * n][2 * hf] * f, o[mt][2 * n + 1][2 * hf] * f);
            const float2 y = make_float2(o[mt][2 * n][2 * hf + 1] * f, o[mt][2 * n + 1][2 * hf + 1] * f);
            *reinterpret_cast<uint2*>(to + n * 16) = a.type == IBWD_BF16
                ? make_uint2(pack2_of(x, __nv_bfloat16{}), pack2_of(y, __nv_bfloat16{}))
                : make_uint2(pack2_of(x, __half{}), pack2_of(y, __half{}));
          }
          if (a.lse && j == 0) a.lse[row] = l2 == 0.f ? -INFINITY : (tm[mt][hf] + log2f(l2)) * 0.69314718055994531f;
        } else {
          float* to = parts + ((long long)(blockIdx.x * 2 + (begun ? 1 : 0)) * ROWS + r) * part_row(D);
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
            *reinterpret_cast<float4*>(to + n * 16 + 4 * j) = make_float4(
                o[mt][2 * n][2 * hf], o[mt][2 * n + 1][2 * hf], o[mt][2 * n][2 * hf + 1], o[mt][2 * n + 1][2 * hf + 1]);
          if (j == 0) *reinterpret_cast<float4*>(to + D) = make_float4(tm[mt][hf], tl[mt][hf], tb[mt][hf], 0.f);
        }
      }
  };

  // ------------------------------------------------------- one step of a warp
  auto compute = [&](const unsigned char* st, unsigned mask) {
    const int first = c.tile * kTile + warp * 16;
    const float* ksc = reinterpret_cast<const float*>(st + 2 * kBytes);
    const float* vsc = ksc + 16;
    float sc[MT][2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
      const int r = nt * 8 + (lane >> 2);
#pragma unroll
      for (int k = 0; k < kLane; ++k) {
        const int ch = D == 64 ? j : (k >> 1) * 8 + 2 * j + (k & 1);
        const uint4 w4 = *reinterpret_cast<const uint4*>(st + stage_at<D>(r, ch));
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t b0, b1;
          adjacent<INT8>(w[g], b0, b1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma_f16(sc[mt][nt], q[mt][k * 4 + g], b0, b1);
        }
      }
    }
    // this lane's positions of the 16: 2j, 2j + 1, 8 + 2j, 9 + 2j
    float ks[2][2], lv[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const float2 x = *reinterpret_cast<const float2*>(ksc + nt * 8 + 2 * j), y = *reinterpret_cast<const float2*>(vsc + nt * 8 + 2 * j);
      ks[nt][0] = x.x;
      ks[nt][1] = x.y;
      lv[nt][0] = __log2f(y.x);
      lv[nt][1] = __log2f(y.y);
    }
    const bool full = mask == 0xFFFFu && (SEL || first + 16 <= lim_min);
    uint32_t p[MT][4];
    bool moved = false;
    float shift[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float y[4], z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int nt = i >> 1, e = i & 1, t = nt * 8 + 2 * j + e;
          y[i] = sc[mt][nt][hf * 2 + e] * (qs[mt][hf] * ks[nt][e]);
          z[i] = y[i] + lv[nt][e];
          if (!full && !((mask >> t & 1) && (SEL || first + t < lim[mt][hf]))) y[i] = z[i] = -INFINITY;
        }
        const float mn = fmaxf(m[mt][hf], quad_max(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]))));
        const float bn = fmaxf(big[mt][hf], quad_max(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]))));
        const float mb = basis(mn), bb = basis(bn) - kUnit;
        float add = 0.f, w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          add += ex2(y[i] - mb);
          w[i] = ex2(z[i] - bb);
        }
        sum[mt][hf] = fmaf(sum[mt][hf], ex2(m[mt][hf] - mb), add);
        shift[mt][hf] = ex2(big[mt][hf] - basis(bn));
        moved = moved || bn != big[mt][hf];
        m[mt][hf] = mn;
        big[mt][hf] = bn;
        p[mt][hf] = half_pair(w[0], w[1]);
        p[mt][2 + hf] = half_pair(w[2], w[3]);
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][i][e] *= shift[mt][e >> 1];
    }
    // values: 16 dimensions a pair of n-tiles, the even ones and the odd ones
    const unsigned char* sv = st + kBytes;
    const int vr = (lane & 7) + (lane >> 3 & 1) * 8, vc = lane >> 4;
    auto values = [&](int i, uint32_t (&b)[4][2]) {  // dimensions 32 i on
      uint32_t w[4];
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(smem_u32(sv + stage_at<D>(vr, 2 * i + vc)))
                   : "memory");
      alternate<INT8>(w[0], b[0][0], b[1][0]);
      alternate<INT8>(w[1], b[0][1], b[1][1]);
      alternate<INT8>(w[2], b[2][0], b[3][0]);
      alternate<INT8>(w[3], b[2][1], b[3][1]);
    };
    if (!INT8 && !SEL && !full) {
      // A NaN that some rows see and others do not: its 0 weight would not keep it out of the others. One position at a time then.
      bool nan = false;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(sv + (i * 32 + lane) * 16);
        const uint32_t x = ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
                           ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
        nan = nan || (x & 0x80808080u);
      }
      if (__any_sync(0xffffffffu, nan)) {
#pragma unroll 1
        for (int t = 0; t < 16; ++t) {
          const uint32_t keep = (t >> 1 & 3) != j ? 0u : t & 1 ? 0xFFFF0000u : 0xFFFFu;
          const uint32_t lo = t < 8 ? keep : 0u, hi = t < 8 ? 0u : keep;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t b[4][2];
            values(i, b);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const uint32_t one[4] = {p[mt][0] & lo, p[mt][1] & lo, p[mt][2] & hi, p[mt][3] & hi};
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(x, one, b[n][0] & lo, b[n][1] & hi);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if ((mask >> t & 1) && first + t < lim[mt][e >> 1]) o[mt][4 * i + n][e] += x[e];
              }
          }
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t b[4][2];
      values(i, b);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mma_f16(o[mt][4 * i + n], p[mt], b[n][0], b[n][1]);
    }
  };

  // -------------------------------------------------------------------- loop
  enter_item();
  int stage = 0;
  for (long long t = t0; t < t1; ++t) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    load(stage == 0 ? STAGES - 1 : stage - 1);
    look_up();
    const unsigned char* st = ring + stage * kStage;
    const unsigned mask = *reinterpret_cast<const unsigned*>(st + 2 * kBytes + 128);
    if (mask) compute(st, mask);
    look_up_page();
    if (++stage == STAGES) stage = 0;
    const bool ends = c.tile + 1 == c.tiles;
    if (ends || t + 1 == t1) leave_item(ends && begun);
    if (t + 1 < t1) {
      if (c.step(a)) {
        begun = true;
        enter_item();
      }
    }
  }
  griddep_launch_dependents();
}

// Joins the parts of items that lie in several blocks: x the block that ends
// one, y four of its rows, four warps a row. 456 parts of one item, the most there
// are, cost their bytes over 4 to 8 SMs.
template <int D, int ROWS>
__global__ void __launch_bounds__(512) attn_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  constexpr int V = D / 32;
  __shared__ float acc[4][4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp & 3;
  griddep_wait();
  const JoinRecord rec = static_cast<const JoinRecord*>(a.work)[blockIdx.x];
  const int r = blockIdx.y * 4 + (warp >> 2), R = rec.row + r;
  if (!rec.valid || rec.row + (int)blockIdx.y * 4 >= rec.rows) return;
  const float* parts = reinterpret_cast<const float*>(static_cast<const JoinRecord*>(a.work) + kAttnGrid);
  const int n = (int)blockIdx.x - rec.first + 1;
  auto part = [&](int i) { return parts + ((long long)((rec.first + i) * 2 + (i == 0)) * ROWS + r) * part_row(D); };
  float m = -INFINITY, big = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  const bool on = R < rec.rows;
  if (on) {
    for (int i = lane; i < n; i += 32) {
      const float4 st = *reinterpret_cast<const float4*>(part(i) + D);
      m = fmaxf(m, st.x);
      big = fmaxf(big, st.z);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, w));
    }
    for (int i = lane; i < n; i += 32) {
      const float4 st = *reinterpret_cast<const float4*>(part(i) + D);
      l += st.y * ex2(st.x - basis(m));
    }
    l = warp_sum(l);
#pragma unroll 8
    for (int i = sub; i < n; i += 4) {
      const float* p = part(i);
      const float f = ex2(p[D + 2] - basis(big));
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(p[e * 32 + lane], f, o[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[warp >> 2][sub][e * 32 + lane] = o[e];
  }
  __syncthreads();
  if (!on || sub) return;
  const float f = l == 0.f ? 0.f : ex2(big - kUnit - basis(m)) / l;
  const int i = R / a.group;
  const long long row = (long long)(rec.token + i) * a.heads * a.group + rec.head * a.group + R - i * a.group;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int d = e * 32 + lane;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += acc[warp >> 2][w][d];
    v *= f;
    if (a.type == IBWD_BF16)
      static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(v);
    else
      static_cast<__half*>(a.out)[row * D + d] = __float2half_rn(v);
  }
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int D, int MT, bool INT8, bool SEL>
cudaError_t attn_launch(const CacheAttnArgs& a, cudaStream_t st) {
  constexpr int STAGES = D == 256 ? 2 : D == 128 ? 4 : 6, BLOCKS = 2;
  constexpr size_t bytes = 4 * STAGES * (2 * 16 * D + 160) + (4 * 16 * MT * 3 + 16) * 4 + 2 * 16 * (D + 4) * 4;
  static std::atomic<size_t> done[64];
  const auto kern = attn_kernel<D, MT, INT8, SEL, STAGES, BLOCKS>;
  cudaError_t e = raise_smem(reinterpret_cast<const void*>(kern), bytes, done);
  if (e != cudaSuccess) return e;
  const int grid = a.num_sms * BLOCKS < kAttnGrid ? a.num_sms * BLOCKS : kAttnGrid;
  const bool vec = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.q_token % 8 == 0 && a.q_head % 8 == 0;
  e = launch_ex(kern, grid, kAttnThreads, bytes, st, false, a, vec);
  if (e != cudaSuccess) return e;
  return launch_ex(attn_join_kernel<D, 16 * MT>, dim3(grid, 4 * MT), 512, 0, st, true, a);
}

template <int D>
cudaError_t attn_launch_of(const CacheAttnArgs& a, cudaStream_t st) {
  // rows of a KV head's queries, on average
  const long long each = a.select || !a.seqs.cu ? 1 : (a.seqs.tokens + a.seqs.batch - 1) / a.seqs.batch;
  const bool wide = D <= 128 && each * a.group > 16;
  auto go = [&](auto mt, auto int8) {
    constexpr int MT = decltype(mt)::value;
    constexpr bool I = decltype(int8)::value;
    return a.select ? attn_launch<D, MT, I, true>(a, st) : attn_launch<D, MT, I, false>(a, st);
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, D <= 128 ? 2 : 1>;
  if (a.code == IBWD_INT8) return wide ? go(Two{}, std::true_type{}) : go(One{}, std::true_type{});
  return wide ? go(Two{}, std::false_type{}) : go(One{}, std::false_type{});
}

}  // namespace ibwd
