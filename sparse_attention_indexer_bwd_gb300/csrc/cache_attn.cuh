// Attention over the paged 8-bit cache, for one or a few query tokens a
// sequence:
//   s_t = scale q . k_t,  p = softmax(s),  out = sum p_t v_t,  lse = log sum exp(s_t).
//
// Bound by the codes' bytes, 2 D a token and KV head, as long as a KV head's
// queries are few: a row tile is 16 or 32 rows (query tokens x heads of the
// group) of a KV head, 16 of heads of 256, and each code is read and converted
// once for a row tile: once where the rows are no more, twice for 64. Of 32x16384
// positions of 8 heads 4 rows take 164 us (97 % of the copy rate), 32 rows 310.
//
// The work is a list of tiles of 128 positions (64 for heads of 256; sequences, KV heads, row tiles,
// positions, in that order), cut into equal runs, one a block, wherever that
// falls, an item of any length counted as two tiles more: lengths are read on the
// device, so ragged batches and single long sequences fill the SMs alike. A block
// joins its four warps at the end of an item (a row tile of a KV head of a
// sequence); an item that lies in several blocks is joined by a second kernel,
// launched behind the first's blocks as they leave, in the order of the blocks.
//
// A warp works alone on 32 positions of a tile (16 where heads are 256 wide):
// cp.async brings their codes to its own ring of stages, mma.sync takes them as
// fp16 (each code, e4m3 or int8, is exact there). The contraction over D runs in
// an order that gives a lane 16 contiguous codes of a key, the same for the
// query; ldmatrix transposes values by bytes. e4m3 keys straight into mma.sync,
// against a query taken apart into e4m3 terms, took longer (157 us for 356 MB).
// tcgen05 would want 128 rows of queries and the codes written to shared memory
// once more in fp16: with 4 to 32 rows its tiles would be mostly padding.
//
// Two running maxima a row: m of the logits (base 2) for the sum l, and M of
// logit - m + log2(|scale| of the value's block), which is what the outputs' unit
// follows, so that a weight has 11 bits relative to the largest contribution
// whatever the blocks' scales are. M counts from m, since log2(scale) beside a
// large logit would be rounded at that one's size. Weights are kept in units of 2^-15, at most
// 2^15 in fp16: they lose bits only below 2^-29 of the largest and vanish below 2^-39.
// A scale below 2^-111 counts as that in M, so that 2^(15 - M) and its inverse are numbers.
#pragma once
#include "cache.h"
#include "elem.cuh"
#include "indexer_cache.h"
#include "kcommon.cuh"
#include "packed.cuh"
#include "train.h"

#include <climits>
#include <type_traits>

namespace ibwd {

constexpr int kAttnThreads = 128;  // four warps
constexpr int kAttnGrid = 456;     // blocks at most, which is what the workspace holds
constexpr float kUnit = 15.f;      // log2 of the largest weight in fp16
constexpr float kLeast = -111.f;   // log2 of a scale at least, in an outputs' unit
constexpr int kItemCost = 2;       // what beginning and ending an item costs, in tiles

// What a block leaves for the join: the item that it ends without having begun it.
struct JoinRecord {
  int valid, first;  // the first block of the item
  int token, row;    // its first query token, the tile's first row
  int rows, head;    // rows of the KV head's queries, the KV head
  int pad[2];
};

// Floats of one partial result's row: outputs in units of 2^(m + M - 15), m, l, M.
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
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
  return r;
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
// What m is where nothing is seen yet: a number, so that differences are none of infinities.
constexpr float kNone = -3.402823466e38f;
// A unit that counts from maximum `m`, as it counts from the larger maximum `to`.
__device__ __forceinline__ float counted(float unit, float m, float to) { return unit + (m - to); }

// Where 16 bytes of a stage's row lie: ldmatrix takes eight rows at once, and a
// lane's quarter of a key two, without a bank conflict. Stages begin on 256
// bytes, so that another chunk of the row is an exclusive or away, and 16 rows
// further 16 D bytes: a step's addresses are few.
template <int D>
__device__ __forceinline__ uint32_t stage_at(int row, int chunk) {
  return row * D + ((chunk ^ (D == 64 ? row >> 1 & 3 : row & 7)) << 4);
}

// Tiles of `len` positions, up to the largest int; one where there are none.
template <int TILE>
__device__ __forceinline__ int tiles_for(int len) {
  return (max(len, 1) - 1) / TILE + 1;
}

// The items in their order, and the tiles of the current one.
template <int ROWS, int TILE, bool SEL>
struct Cursor {
  int b;        // sequence; SEL: the query token
  int head, rt;
  int tile, tiles;
  int row_tiles, rows;  // row tiles and rows of a KV head
  int token;            // first query token
  int len;              // positions held; SEL: places of the list
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
      seen = n ? (int)max(-(1ll << 30), (long long)s.lens[b] - n + 1) : 0;  // (n is at most 2^27)
      rows = (int)min((long long)n * a.group, 1ll << 30);
    }
    row_tiles = (rows + ROWS - 1) / ROWS;
    tiles = tiles_for<TILE>(len);
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

// What sequence b costs, in tiles.
template <int ROWS, int TILE>
__device__ __forceinline__ long long tiles_of(const CacheAttnArgs& a, int b) {
  const CacheSeqs& s = a.seqs;
  const long long n = s.begin(b + 1) - s.begin(b);
  if (n <= 0) return 0;
  return (n * a.group + ROWS - 1) / ROWS * a.heads * (kItemCost + tiles_for<TILE>(s.length(b)));
}

// Groups of 16 positions in a warp's step.
constexpr int attn_subs(int D) { return D == 256 ? 1 : 2; }
// Bytes of a stage: keys, values, a mask, and the scales of each group (SEL: each position).
constexpr int attn_stage(int D, bool sel) { return (attn_subs(D) * (32 * D + (sel ? 128 : 0)) + 32 + 255) / 256 * 256; }

template <int D, int MT, bool INT8, bool SEL, int STAGES, int BLOCKS>
__global__ void __launch_bounds__(kAttnThreads, BLOCKS) attn_kernel(const __grid_constant__ CacheAttnArgs a, bool vec, long long most_tiles) {
  constexpr int ROWS = 16 * MT, kRowChunks = D / 16;
  constexpr int SUBS = attn_subs(D), STEP = 16 * SUBS, kTile = 4 * STEP;  // positions of a warp's step, of a block's
  constexpr int kBytes = STEP * D, kStage = attn_stage(D, SEL);
  constexpr int kLane = D / 64;             // 16-byte chunks of a key that a lane takes
  extern __shared__ __align__(256) unsigned char smem[];
  __shared__ long long scan[5];
  __shared__ int found_b;
  __shared__ long long found_rest;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane & 3;
  const CacheSeqs& s = a.seqs;
  griddep_launch_dependents();  // the join's blocks come in as these leave

  // ------------------------------------------------- this block's run of tiles
  using Place = Cursor<ROWS, kTile, SEL>;
  Place c;
  long long total, t0, t1;
  long long blocks;  // that have tiles: at least one each, since the join takes a part of each
  c.head = c.rt = c.tile = 0;
  if (SEL) {
    const int from = s.cu ? s.begin(0) : 0;  // (rows before the first sequence are nobody's)
    const int tokens = max(0, (s.cu ? s.begin(s.batch) : (int)s.tokens) - from);
    const long long each = (long long)((a.group + ROWS - 1) / ROWS) * a.heads * (kItemCost + tiles_for<kTile>(a.kept));
    total = each * tokens;
    blocks = min((long long)gridDim.x, total);
    t0 = blockIdx.x < blocks ? total * blockIdx.x / blocks : 0;
    t1 = blockIdx.x < blocks ? total * (blockIdx.x + 1) / blocks : 0;
    c.b = (int)(t0 / each);
    found_rest = t0 - c.b * each;  // (alike in all threads)
    c.b += from;
  } else {
    const int per = (s.batch + kAttnThreads - 1) / kAttnThreads;
    const int b0 = min((int)threadIdx.x * per, s.batch), b1 = min(b0 + per, s.batch);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += tiles_of<ROWS, kTile>(a, b);
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
    // offsets that fall count tokens several times: of such a call, whose results are undefined, there is no more to do than
    // of any other
    if (total > most_tiles) total = 0;
    blocks = min((long long)gridDim.x, total);
    t0 = blockIdx.x < blocks ? total * blockIdx.x / blocks : 0;
    t1 = blockIdx.x < blocks ? total * (blockIdx.x + 1) / blocks : 0;
    if (t0 >= upto - sum && t0 < upto) {
      long long rest = t0 - (upto - sum);
      int b = b0;
      for (; b < b1; ++b) {
        const long long n = tiles_of<ROWS, kTile>(a, b);
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
    return;
  }
  if (SEL) __syncthreads();
  long long rest = found_rest;
  c.enter(a);
  const int units = (int)(t1 - t0);
  int skipped;  // of the first item's own cost
  {
    const long long per_tile = c.tiles + kItemCost, per_head = c.row_tiles * per_tile;
    c.head = (int)(rest / per_head);
    rest -= c.head * per_head;
    c.rt = (int)(rest / per_tile);
    rest -= c.rt * per_tile;
    c.tile = (int)max(0ll, rest - kItemCost);
    skipped = (int)max(0ll, kItemCost - rest);
  }
  if (threadIdx.x == 0) {
    const long long begin = t0 - rest + kItemCost;  // of the item's first tile
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
  if (units <= skipped) return;

  // ------------------------------------------------------------------- loads
  unsigned char* ring = smem + warp * (STAGES * kStage);
  uint4* queries = reinterpret_cast<uint4*>(smem + 4 * STAGES * kStage);  // [MT][D / 16][32] fragments
  float* stats = reinterpret_cast<float*>(queries + MT * D * 2);          // [4][ROWS][3]
  const int P = 1 << s.page_log;
  // An item's queries on their way to L2, before they are asked for.
  auto fetch_queries = [&](const Place& p) {
    const int r = p.rt * ROWS + lane, i = r / a.group;
    if (warp || lane >= ROWS || r >= p.rows) return;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (long long)(p.token + i) * a.q_token +
                        (long long)(p.head * a.group + r - i * a.group) * a.q_head;
#pragma unroll
    for (int d = 0; d < D; d += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + d));
  };
  fetch_queries(c);
  // Two steps are on their way before a load: its pages (SEL: its places of the list) are looked up, then their scales (the
  // pages) are; each answer has a step's time to arrive.
  Place n = c;                  // the step that is looked up
  int ahead = units - skipped;  // of the run, from there on
  int found[SUBS];              // dense: the pages of its positions; SEL: this lane's position
  // what the next load takes. Dense: its first position, and of each 16 positions their page and its scales; SEL: this
  // lane's position and its page
  bool more = false;
  int at = 0, head = 0, len = 0, page[SUBS];
  float next_k[SUBS], next_v[SUBS];
#pragma unroll
  for (int i = 0; i < SUBS; ++i) {
    page[i] = found[i] = -1;
    next_k[i] = next_v[i] = 0.f;
  }
  auto look_up = [&]() {
    if (ahead <= 0) return;
    const int first = n.tile * kTile + warp * STEP;
    if (SEL) {
      found[0] = lane < STEP && first + lane < a.kept ? a.select[(long long)n.token * a.kept + first + lane] : -1;
    } else {
#pragma unroll
      for (int i = 0; i < SUBS; ++i) found[i] = first + 16 * i < n.len ? s.page_at(n.seq, first + 16 * i) : -1;
    }
  };
  auto settle = [&]() {
    more = ahead > 0;
    if (!more) return;
    head = n.head;
    len = n.len;
    if (SEL) {
      at = found[0];
      page[0] = at >= 0 && at < n.seen ? s.page_at(n.seq, at) : -1;
    } else {
      at = n.tile * kTile + warp * STEP;
#pragma unroll
      for (int i = 0; i < SUBS; ++i) {
        page[i] = found[i];
        if (page[i] >= 0) {
          const long long block = (long long)page[i] * a.heads + head;
          next_k[i] = a.k_scale[block];
          next_v[i] = a.v_scale[block];
        }
      }
    }
    if (--ahead > 0 && n.tile + 1 == n.tiles) ahead -= kItemCost;
    if (ahead > 0 && n.step(a)) fetch_queries(n);
  };
  const uint32_t put = stage_at<D>(lane / kRowChunks, lane % kRowChunks);
  auto load = [&](int stage) {
    if (more) {
      unsigned char* to = ring + stage * kStage;
      const uint32_t to32 = smem_u32(to);
      // this lane's chunk of the 512 bytes after n times 512
      auto place = [&](int n) {
        const int turn = D == 64 ? 0 : D == 128 ? (n & 1) * 64 : (2 * n & 7) << 4;
        return ((to32 + put) ^ turn) + n * 512;
      };
      unsigned mask;
      if (SEL) {
        mask = __ballot_sync(0xffffffffu, page[0] >= 0);
        const long long block = (long long)page[0] * a.heads + head;
        const long long row = page[0] >= 0 ? (block << s.page_log) + (at & (P - 1)) : 0;
        if (mask) {
#pragma unroll
          for (int i = 0; i < SUBS * kRowChunks / 2; ++i) {
            const int r = (i * 32 + lane) / kRowChunks;
            const long long src = __shfl_sync(0xffffffffu, row, r) * D + (lane % kRowChunks) * 16;
            const uint32_t bytes = mask >> r & 1 ? 16u : 0u;
            const uint32_t dst = place(i);
            cp_async16(dst, static_cast<const uint8_t*>(a.k) + src, bytes);
            cp_async16(dst + kBytes, static_cast<const uint8_t*>(a.v) + src, bytes);
          }
          if (lane < STEP) {
            const bool on = page[0] >= 0;
            cp_async4(to32 + 2 * kBytes + 32 + 4 * lane, a.k_scale + (on ? block : 0), on ? 4u : 0u);
            cp_async4(to32 + 2 * kBytes + 32 + 4 * (STEP + lane), a.v_scale + (on ? block : 0), on ? 4u : 0u);
          }
        }
      } else {
        const int count = len - at;
        mask = count >= 32 ? 0xFFFFFFFFu : count <= 0 ? 0u : (1u << count) - 1u;
        if (SUBS == 1) mask &= 0xFFFFu;
#pragma unroll
        for (int i = 0; i < SUBS; ++i) {
          if (page[i] < 0) mask &= ~(0xFFFFu << (16 * i));
          const unsigned part = mask >> (16 * i) & 0xFFFFu;
          if (!part) continue;
          // sixteen rows side by side in the cache
          const long long row = (((long long)page[i] * a.heads + head) << s.page_log) + ((at + 16 * i) & (P - 1));
          const uint8_t *k = static_cast<const uint8_t*>(a.k) + row * D + lane * 16, *v = static_cast<const uint8_t*>(a.v) + row * D + lane * 16;
          if (part == 0xFFFFu) {
#pragma unroll
            for (int n = 0; n < kRowChunks / 2; ++n) {
              const uint32_t dst = place(i * kRowChunks / 2 + n);
              cp_async16(dst, k + n * 512, 16u);
              cp_async16(dst + kBytes, v + n * 512, 16u);
            }
          } else {
#pragma unroll
            for (int n = 0; n < kRowChunks / 2; ++n) {
              const int r = (n * 32 + lane) / kRowChunks;
              const uint32_t dst = place(i * kRowChunks / 2 + n);
              const uint32_t bytes = part >> r & 1 ? 16u : 0u;
              cp_async16(dst, k + n * 512, bytes);
              cp_async16(dst + kBytes, v + n * 512, bytes);
            }
          }
        }
      }
      if (lane == 0) {
        *reinterpret_cast<unsigned*>(to + 2 * kBytes) = mask;
        if (!SEL) *reinterpret_cast<float4*>(to + 2 * kBytes + 16) = make_float4(next_k[0], next_v[0], next_k[SUBS - 1], next_v[SUBS - 1]);
      }
    }
    cp_async_commit();
  };
  look_up();
  settle();
  look_up();
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    load(i);
    settle();
    look_up();
  }

  // ------------------------------------------------------------------- items
  float qs[MT][2], m[MT][2], big[MT][2], sum[MT][2];
  int lim[MT][2], lim_min = 0;
  float o[MT][D / 8][4];
  bool begun = c.tile == 0;  // the segment at hand holds its item's first tile

  // The item's queries as fragments in shared memory, the same for all warps: each writes a quarter.
  auto enter_item = [&]() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint4 raw[2][kLane][2];
      float down[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = c.rt * ROWS + mt * 16 + hf * 8 + (lane >> 2);
        const bool on = r < c.rows;
        const int i = r / a.group;
        lim[mt][hf] = SEL ? 0 : on ? c.seen + i : -1;
        const uint16_t* p = static_cast<const uint16_t*>(a.q) +
                            (on ? (long long)(c.token + i) * a.q_token + (long long)(c.head * a.group + r - i * a.group) * a.q_head : 0);
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
          const int ch = D == 64 ? j : (k >> 1) * 8 + 2 * j + (k & 1);
          raw[hf][k][0] = raw[hf][k][1] = make_uint4(0, 0, 0, 0);
          if (on) {
            if (vec) {
              raw[hf][k][0] = *reinterpret_cast<const uint4*>(p + ch * 16);
              raw[hf][k][1] = *reinterpret_cast<const uint4*>(p + ch * 16 + 8);
            } else {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = (uint32_t)p[ch * 16 + 2 * e] | (uint32_t)p[ch * 16 + 2 * e + 1] << 16;
              raw[hf][k][0] = make_uint4(w[0], w[1], w[2], w[3]);
              raw[hf][k][1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      auto two = [&](uint32_t w) { return a.type == IBWD_BF16 ? unpack2(w, __nv_bfloat16{}) : unpack2(w, __half{}); };
      auto word = [&](int hf, int k, int e) {
        const uint4 x = raw[hf][k][e >> 2];
        return (e & 3) == 0 ? x.x : (e & 3) == 1 ? x.y : (e & 3) == 2 ? x.z : x.w;
      };
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < kLane; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = two(word(hf, k, e));
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        amax = quad_max(amax);
        // The row in units of 2^e with its largest entry in [1, 2). An infinite query gives NaN.
        const int e = min((int)(__float_as_uint(amax) >> 23) - 127, 126);
        const bool none = amax == 0.f || e < -126;
        down[hf] = none ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23);
        qs[mt][hf] = (none ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23)) * a.scale_log2;
        if (amax == INFINITY) qs[mt][hf] = __uint_as_float(0x7FC00000u);
        m[mt][hf] = kNone;
        big[mt][hf] = kLeast;
        sum[mt][hf] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < kLane; ++k)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (warp == g) {  // words 2 g, 2 g + 1 of a chunk are a step of 16 dimensions
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = two(word(e & 1, k, 2 * g + (e >> 1)));
              w[e] = half_pair(f.x * down[e & 1], f.y * down[e & 1]);
            }
            queries[(mt * (D / 16) + k * 4 + g) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
          }
    }
    lim_min = c.seen + c.rt * ROWS / a.group;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
    __syncthreads();
  };

  // Joins the warps' results of the segment: to `out` where it is the whole item, else to the block's parts. They meet in
  // the stages that were just used, which nothing is loaded into before the last barrier.
  auto leave_item = [&](bool whole, int stage) {
    constexpr int DC = D > 128 ? 128 : D;  // dimensions at a time: 16 rows of them in fp32 fill a stage
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
    // 8-byte units of a row, turned by the row so that eight rows lie in different banks
    auto at = [&](int w, int row, int unit) {
      return reinterpret_cast<float*>(smem + (w * STAGES + stage) * kStage + row * DC * 4 + ((unit ^ (4 * (row & 7))) << 3));
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int d0 = 0; d0 < D; d0 += DC) {
        if (mt || d0) __syncthreads();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          if (mt * 16 + hf * 8 < c.rows - c.rt * ROWS)
#pragma unroll
          for (int i = 0; i < DC / 8; ++i)
            *reinterpret_cast<float2*>(at(warp, hf * 8 + (lane >> 2), i * 4 + j)) =
                make_float2(o[mt][d0 / 8 + i][2 * hf], o[mt][d0 / 8 + i][2 * hf + 1]);
        __syncthreads();
        // a warp a row
#pragma unroll 1
        for (int row = warp; row < 16; row += 4) {
          const int r = mt * 16 + row, R = c.rt * ROWS + r;
          if (R >= c.rows) break;
          const float* p = stats + r * 3;
          float mm = kNone, bb = kNone, ll = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            mm = fmaxf(mm, p[w * ROWS * 3]);
            bb = fmaxf(bb, p[w * ROWS * 3] + p[w * ROWS * 3 + 2]);
          }
          bb = fmaxf(bb - mm, kLeast);  // (rounded, but any unit near the largest serves in fp32)
          constexpr int V = DC / 32;
          float x[V];
#pragma unroll
          for (int e = 0; e < V; ++e) x[e] = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            ll = fmaf(p[w * ROWS * 3 + 1], ex2(p[w * ROWS * 3] - mm), ll);
            const float f = ex2(counted(p[w * ROWS * 3 + 2], p[w * ROWS * 3], mm) - bb);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const float2 v = *reinterpret_cast<const float2*>(at(w, row, (lane * V + e) / 2));
              x[e] = fmaf(v.x, f, x[e]);
              x[e + 1] = fmaf(v.y, f, x[e + 1]);
            }
          }
          if (whole) {
            const int i = R / a.group;
            const long long out_row = (long long)(c.token + i) * a.heads * a.group + c.head * a.group + R - i * a.group;
            const float f = ll == 0.f ? 0.f : 1.f / ll, unit = ex2(bb - kUnit);
            uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + out_row * D + d0 + lane * V);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const float2 v = make_float2(x[e] * f * unit, x[e + 1] * f * unit);
              to[e / 2] = a.type == IBWD_BF16 ? pack2_of(v, __nv_bfloat16{}) : pack2_of(v, __half{});
            }
            if (a.lse && lane == 0 && d0 == 0) a.lse[out_row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f;
          } else {
            float* to = parts + ((long long)(blockIdx.x * 2 + (begun ? 1 : 0)) * ROWS + r) * part_row(D);
#pragma unroll
            for (int e = 0; e < V; e += 2) *reinterpret_cast<float2*>(to + d0 + lane * V + e) = make_float2(x[e], x[e + 1]);
            if (lane == 0 && d0 == 0) *reinterpret_cast<float4*>(to + D) = make_float4(mm, ll, bb, 0.f);
          }
        }
      }
    __syncthreads();
  };

  // ------------------------------------------------------- one step of a warp
  const uint32_t key_at = stage_at<D>(4 * (lane >> 3) + (lane >> 2 & 1), D == 64 ? j : 2 * j);
  const uint32_t value_at = stage_at<D>(lane & 15, lane >> 4);
  auto compute = [&](const unsigned char* st) {
    const int first = c.tile * kTile + warp * STEP;
    const unsigned mask = *reinterpret_cast<const unsigned*>(st + 2 * kBytes);
    if (!mask) return;
    // Scores of 16 x STEP: column n of n-tile t is position 16 (t / 2) + 4 (n / 2) + (n & 1) + 2 (t & 1), so that a lane has
    // four positions side by side of each 16, as the values' fragments want them.
    constexpr int NT = 2 * SUBS;
    float sc[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
    const uint32_t keys = smem_u32(st) + key_at;
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      uint4 w[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t turn = (((k >> 1) * 8 + (k & 1)) << 4) ^ (nt & 1 ? (D == 64 ? 16 : 32) : 0);
        w[nt] = ld_shared16((keys ^ turn) + (16 * (nt >> 1) + 2 * (nt & 1)) * D);
      }
      uint32_t b[4][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        adjacent<INT8>(w[nt].x, b[0][nt][0], b[0][nt][1]);
        adjacent<INT8>(w[nt].y, b[1][nt][0], b[1][nt][1]);
        adjacent<INT8>(w[nt].z, b[2][nt][0], b[2][nt][1]);
        adjacent<INT8>(w[nt].w, b[3][nt][0], b[3][nt][1]);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint4 f = queries[(mt * (D / 16) + k * 4 + g) * 32 + lane];
          const uint32_t q[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(sc[mt][nt], q, b[g][nt][0], b[g][nt][1]);
        }
      }
    }
    // this lane's positions: 16 u + 4 j + e. The scales of each 16 of them, or (SEL) their own.
    float ks[SUBS][SEL ? 4 : 1], vs[SUBS][SEL ? 4 : 1], lv[SUBS][SEL ? 4 : 1];
    float most[SUBS];  // of lv
    if (SEL) {
      const float* own = reinterpret_cast<const float*>(st + 2 * kBytes + 32) + 4 * j;
#pragma unroll
      for (int u = 0; u < SUBS; ++u) {
        const float4 x = *reinterpret_cast<const float4*>(own + 16 * u), y = *reinterpret_cast<const float4*>(own + STEP + 16 * u);
        const float xx[4] = {x.x, x.y, x.z, x.w}, yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < (SEL ? 4 : 1); ++e) {
          ks[u][e] = xx[e];
          vs[u][e] = yy[e];
          lv[u][e] = fmaxf(__log2f(fabsf(yy[e])), kLeast);
        }
        most[u] = fmaxf(fmaxf(lv[u][0], lv[u][SEL ? 1 : 0]), fmaxf(lv[u][SEL ? 2 : 0], lv[u][SEL ? 3 : 0]));
      }
    } else {
      const float4 x = *reinterpret_cast<const float4*>(st + 2 * kBytes + 16);
#pragma unroll
      for (int u = 0; u < SUBS; ++u) {
        ks[u][0] = u ? x.z : x.x;
        vs[u][0] = u ? x.w : x.y;
        most[u] = lv[u][0] = fmaxf(__log2f(fabsf(vs[u][0])), kLeast);
      }
    }
    const int here = c.rows - c.rt * ROWS;  // rows of this tile, and on
    constexpr unsigned kAll = SUBS == 2 ? 0xFFFFFFFFu : 0xFFFFu;
    const bool full = mask == kAll && (SEL || first <= lim_min - STEP);
    // Half of a tile may have no rows (KV heads of four, int8: 180 us where it went through the softmax as well, 172 without).
    auto empty = [&](int hf) { return MT == 1 && hf && here <= 8; };
    // The logit of a row's position e of a lane's four in each 16, then less its row's maximum.
    auto y = [&](int mt, int hf, int u, int e) -> float& { return sc[mt][2 * u + (e >> 1)][2 * hf + (e & 1)]; };
    // Whether a contribution may pass its row's unit: by what is there before the step, so that nothing waits for the maxima.
    bool moved = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (empty(hf)) continue;
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
          const float unit = qs[mt][hf] * ks[u][0];
#pragma unroll
          for (int e = 0; e < 4; ++e) y(mt, hf, u, e) *= SEL ? qs[mt][hf] * ks[u][SEL ? e : 0] : unit;
        }
        if (!full) {
#pragma unroll
          for (int u = 0; u < SUBS; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = 16 * u + 4 * j + e;
              if (!((mask >> t & 1) && (SEL || first + t < lim[mt][hf]))) y(mt, hf, u, e) = -INFINITY;
            }
        }
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
          const float t4 = fmaxf(fmaxf(y(mt, hf, u, 0), y(mt, hf, u, 1)), fmaxf(y(mt, hf, u, 2), y(mt, hf, u, 3)));
          top = fmaxf(top, t4);
          moved = moved || t4 - m[mt][hf] + most[u] > big[mt][hf];
        }
        const float mn = fmaxf(m[mt][hf], quad_max(top));
#pragma unroll
        for (int u = 0; u < SUBS; ++u)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 d = add2(make_float2(y(mt, hf, u, e), y(mt, hf, u, e + 1)), both(-mn));
            y(mt, hf, u, e) = d.x;
            y(mt, hf, u, e + 1) = d.y;
          }
        sum[mt][hf] *= ex2(m[mt][hf] - mn);
        big[mt][hf] = counted(big[mt][hf], m[mt][hf], mn);
        m[mt][hf] = mn;
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (empty(hf)) continue;
          float over = -INFINITY;
#pragma unroll
          for (int u = 0; u < SUBS; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) over = fmaxf(over, y(mt, hf, u, e) + lv[u][SEL ? e : 0]);
          const float bn = fmaxf(big[mt][hf], quad_max(over)), shift = ex2(big[mt][hf] - bn);
          big[mt][hf] = bn;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[mt][i][2 * hf] *= shift;
            o[mt][i][2 * hf + 1] *= shift;
          }
        }
    }
    // A weight is its probability 2^(y - m) times its value's scale, in units of 2^(M - 15): in that order, since the last two
    // alone may be beyond fp32. A probability below 2^-126 is 0, whatever its value's scale.
    uint32_t p[MT][SUBS][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (empty(hf)) {
#pragma unroll
          for (int u = 0; u < SUBS; ++u) p[mt][u][hf] = p[mt][u][2 + hf] = 0u;
          continue;
        }
        float2 add = make_float2(0.f, 0.f);
        const float unit = ex2(kUnit - big[mt][hf]);
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 pr = make_float2(ex2(y(mt, hf, u, e)), ex2(y(mt, hf, u, e + 1)));
            add = add2(add, pr);
            const float2 x = mul2(mul2(pr, both(unit)), make_float2(vs[u][SEL ? e : 0], vs[u][SEL ? e + 1 : 0]));
            w[e] = x.x;
            w[e + 1] = x.y;
          }
          if (!full) {  // (an invisible position's scale may be anything)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (y(mt, hf, u, e) == -INFINITY) w[e] = 0.f;
          }
          p[mt][u][hf] = half_pair(w[0], w[1]);
          p[mt][u][2 + hf] = half_pair(w[2], w[3]);
        }
        sum[mt][hf] += add.x + add.y;
      }
    // Values: of 32 dimensions four n-tiles, a lane's four positions side by side.
    const unsigned char* sv = st + kBytes;
    const uint32_t rows = smem_u32(sv) + value_at;
    auto values = [&](int u, int i, uint32_t (&b)[4][2]) {
      uint32_t w[4];
      asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"((rows ^ (32 * i)) + 16 * u * D)
                   : "memory");
#pragma unroll
      for (int n = 0; n < 4; ++n) adjacent<INT8>(w[n], b[n][0], b[n][1]);
    };
    if (!INT8 && !SEL && !full) {
      // A NaN that some rows see and others do not: its 0 weight would not keep it out of the others. One position at a time then.
      bool nan = false;
#pragma unroll
      for (int i = 0; i < STEP * D / 512; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(sv + (i * 32 + lane) * 16);
        const int r = (i * 32 + lane) / kRowChunks;
        const uint32_t x = ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
                           ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
        nan = nan || ((x & 0x80808080u) && (mask >> r & 1));
      }
      if (__any_sync(0xffffffffu, nan)) {
#pragma unroll 1
        for (int t = 0; t < STEP; ++t) {
          if (!(mask >> t & 1)) continue;
          const int u = t >> 4;
          const uint32_t keep = (t >> 2 & 3) != j ? 0u : t & 1 ? 0xFFFF0000u : 0xFFFFu;
          const uint32_t lo = t & 2 ? 0u : keep, hi = t & 2 ? keep : 0u;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t b[4][2];
            values(u, i, b);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                uint32_t one[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) one[e] = (u && SUBS == 2 ? p[mt][SUBS - 1][e] : p[mt][0][e]) & (e < 2 ? lo : hi);
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(x, one, b[n][0] & lo, b[n][1] & hi);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (first + t < lim[mt][e >> 1]) o[mt][4 * i + n][e] += x[e];
              }
          }
        }
        return;
      }
    }
#pragma unroll
    for (int u = 0; u < SUBS; ++u) {
      // (16 positions that nothing was loaded for: what lies there may be any bits)
      if (!(mask >> (16 * u) & 0xFFFFu)) continue;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t b[4][2];
        values(u, i, b);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mma_f16(o[mt][4 * i + n], p[mt][u], b[n][0], b[n][1]);
      }
    }
  };

  // -------------------------------------------------------------------- loop
  enter_item();
  int stage = 0, run = units - skipped;
  while (true) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    load(stage == 0 ? STAGES - 1 : stage - 1);
    settle();
    look_up();
    compute(ring + stage * kStage);
    const bool ends = c.tile + 1 == c.tiles;
    --run;
    if (ends) run -= kItemCost;
    if (ends || run <= 0) leave_item(ends && begun, stage);
    if (run <= 0) break;
    if (++stage == STAGES) stage = 0;
    if (c.step(a)) {
      begun = true;
      enter_item();
    }
  }
}

// Joins the parts of items that lie in several blocks: x `per` of the blocks that
// may end one, y two of its rows. A thread takes the statistics of a part or two,
// while the eight warps' first parts of the outputs are on their way, four of
// each row a warp at once; they meet in shared memory in their order: of a single
// item in all blocks (one sequence of 131072 tokens, one KV head) the parts are
// 600 KB. Several blocks' records a block where rows are many, so that the grid
// is twice what is resident at most: most records end no item (64 selections of 16 rows
// 20.7 us, a record a block 22.8).
template <int D, int ROWS>
__global__ void __launch_bounds__(256, 4) attn_join_kernel(const __grid_constant__ CacheAttnArgs a, int per, int grid) {
  constexpr int V = D / 32, U = D == 256 ? 2 : 4;
  __shared__ float factor[2][kAttnGrid];
  __shared__ float red[2][3][8];
  __shared__ float acc[8][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = blockIdx.y * 2, mine = (int)blockIdx.x * per + lane;
  griddep_wait();
  const JoinRecord* records = static_cast<const JoinRecord*>(a.work);
  const float* parts = reinterpret_cast<const float*>(records + kAttnGrid);
  JoinRecord held{};
  if (lane < per && mine < grid) held = records[mine];
  unsigned todo = __ballot_sync(0xffffffffu, held.valid && held.row + r0 < held.rows);
  for (; todo; todo &= todo - 1) {
    const int from = __ffs(todo) - 1;
    auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, from); };
    const int first = of(held.first), token = of(held.token), top = of(held.row) + r0, head = of(held.head);
    const int n = (int)blockIdx.x * per + from - first + 1, rows = min(2, of(held.rows) - top);
    auto part = [&](int i, int r) { return parts + ((long long)((first + i) * 2 + (i == 0)) * ROWS + r0 + r) * part_row(D); };
    // Parts i, i + 8, .. of a warp (a row beyond the item's as the first). At first as many as there are: most items have few.
    // Then those beyond the last as the last, since a load under a condition is waited for before the next (a single item
    // of 342 parts 37 us, not 29).
    float x[2][U][V];
    auto load = [&](int u, int i) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float* p = part(i, r < rows ? r : 0) + lane;
#pragma unroll
        for (int e = 0; e < V; ++e) asm volatile("ld.global.f32 %0, [%1];" : "=f"(x[r][u][e]) : "l"(p + e * 32));
      }
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (warp + 8 * u < n) load(u, warp + 8 * u);
    constexpr int S = (kAttnGrid + 255) / 256;
    float4 st[2][S];
    float m[2], big[2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const int i = threadIdx.x + 256 * k;
        st[r][k] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        if (i < n && r < rows) st[r][k] = *reinterpret_cast<const float4*>(part(i, r) + D);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m[r] = big[r] = -INFINITY;
#pragma unroll
      for (int k = 0; k < S; ++k) {
        m[r] = fmaxf(m[r], st[r][k].x);
        big[r] = fmaxf(big[r], st[r][k].x + st[r][k].z);
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) {
        m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], w));
        big[r] = fmaxf(big[r], __shfl_xor_sync(0xffffffffu, big[r], w));
      }
      if (lane == 0) {
        red[r][0][warp] = m[r];
        red[r][1][warp] = big[r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        m[r] = fmaxf(m[r], red[r][0][w]);
        big[r] = fmaxf(big[r], red[r][1][w]);
      }
      big[r] = fmaxf(big[r] - m[r], kLeast);  // (as where warps meet)
      float l = 0.f;
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const int i = threadIdx.x + 256 * k;
        l = fmaf(st[r][k].y, ex2(st[r][k].x - m[r]), l);
        if (i < n) factor[r][i] = ex2(counted(st[r][k].z, st[r][k].x, m[r]) - big[r]);
      }
      l = warp_sum(l);
      if (lane == 0) red[r][2][warp] = l;
    }
    __syncthreads();
    float o[2][V];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < V; ++e) o[r][e] = 0.f;
    for (int i = warp; i < n; i += 8 * U) {
      if (i != warp)
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, min(i + 8 * u, n - 1));
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i + 8 * u < n) {
#pragma unroll
            for (int e = 0; e < V; ++e) o[r][e] = fmaf(x[r][u][e], factor[r][i + 8 * u], o[r][e]);
          }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[warp][r][e * 32 + lane] = o[r][e];
    __syncthreads();
    for (int idx = threadIdx.x; idx < rows * D; idx += 256) {
      const int r = idx / D, d = idx - r * D, R = top + r, i = R / a.group;
      const long long row = (long long)(token + i) * a.heads * a.group + head * a.group + R - i * a.group;
      const float mr = r ? m[1] : m[0], br = r ? big[1] : big[0];
      float v = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        v += acc[w][r][d];
        l += red[r][2][w];
      }
      v = l == 0.f ? 0.f : v * (1.f / l) * ex2(br - kUnit);
      if (a.type == IBWD_BF16)
        static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(v);
      else
        static_cast<__half*>(a.out)[row * D + d] = __float2half_rn(v);
      if (a.lse && d == 0) a.lse[row] = l == 0.f ? -INFINITY : (mr + log2f(l)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

template <int D, int MT, bool INT8, bool SEL>
cudaError_t attn_launch(const CacheAttnArgs& a, cudaStream_t st) {
  constexpr int BLOCKS = D * MT <= 128 && (D == 128 || MT == 1) ? 3 : 2, STAGES = D == 64 ? 4 : BLOCKS == 3 ? 2 : 3;
  constexpr size_t bytes = 4 * STAGES * attn_stage(D, SEL) + MT * D * 32 + 4 * 16 * MT * 3 * 4;
  static std::atomic<size_t> done[64];
  const auto kern = attn_kernel<D, MT, INT8, SEL, STAGES, BLOCKS>;
  cudaError_t e = raise_smem(reinterpret_cast<const void*>(kern), bytes, done);
  if (e != cudaSuccess) return e;
  const int grid = a.num_sms * BLOCKS < kAttnGrid ? a.num_sms * BLOCKS : kAttnGrid;
  const bool vec = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.q_token % 8 == 0 && a.q_head % 8 == 0;
  // The tiles of the call at most, with the items' own cost. A block's run of them is an int: the entry point sees to that.
  const long long items = a.select ? (a.group + 16 * MT - 1) / (16 * MT) * a.seqs.tokens
                                   : a.seqs.tokens * a.group / (16 * MT) + (a.seqs.batch < a.seqs.tokens ? a.seqs.batch : a.seqs.tokens);
  const long long places = a.select ? a.kept : (long long)a.seqs.width << a.seqs.page_log;
  const long long most_tiles = items * a.heads * (kItemCost + (places - 1) / (64 * attn_subs(D)) + 1);
  if (most_tiles / grid >= INT_MAX) return cudaErrorInvalidValue;
  // Not launched before the kernel in front has ended: its blocks would take
  // places as that one's leave, unevenly (64 ragged sequences 93 us, not 70).
  e = launch_ex(kern, grid, kAttnThreads, bytes, st, false, a, vec, most_tiles);
  if (e != cudaSuccess) return e;
  // rows that an item can have
  const int rows = (a.select || !a.seqs.cu) && a.group < 16 * MT ? a.group : 16 * MT;
  const int pairs = (rows + 1) / 2, most = 8 * a.num_sms, per = (grid * pairs + most - 1) / most;
  return launch_ex(attn_join_kernel<D, 16 * MT>, dim3((grid + per - 1) / per, pairs), 256, 0, st, true, a, per, grid);
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
