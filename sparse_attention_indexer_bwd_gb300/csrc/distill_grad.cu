// Distillation loss and gradient in one call on sm_103a, each logit read once
// and its gradient written once: bound by HBM.
//
//   p = softmax over the kept slots of teacher / T,  q = softmax of logits / T
//   loss = T^2 sum_j p_j (log p_j - log q[id_j]),
//   dlogits_v = g (q_v - sum_{id_j = v} p_j)
//
// The gradient of a row needs the sum over all of it, so the row has to wait
// somewhere between its two passes.  Read again from L2 it ran at 60 % of HBM
// (4096 rows of 131072 bf16: 503 us); here it stays in shared memory: a block
// of 256 threads holds up to 64 KB of a row, three blocks to an SM, so that
// one loads while another computes and a third writes, and a cluster of
// blocks holds a longer row.  (One block an SM that walks the rows through a
// ring of three such buffers took 732 us: all its warps are in one phase.)
// 4096 rows of 131072 bf16: 371 us, 5.8 TB/s; 16384 of 32768: 330 us, 6.5.
// Two exponentials an element are three quarters of what the SMs' special
// function units give at HBM's rate, so the phases have to overlap well.
//
// The blocks of a cluster meet once, through distributed shared memory: the
// part's statistic and what the loss needs of the kept tokens in it, taken
// relative to the part's own maximum, travel together.
//
// Every sum is joined in a fixed order; results are bitwise reproducible.
#include <cooperative_groups.h>

#include <algorithm>

#include "indexer_train.h"
#include "logits.cuh"

namespace cg = cooperative_groups;

namespace ibwd {
namespace {

constexpr int kGroups = 4;  // copies of a part are taken up in so many steps
template <int NT>
constexpr int kRoom = kGroups * kUnroll * NT;  // vectors of a part that NT threads hold
constexpr int kMaxWarps = 256 / 32;
// Blocks of an SM: registers for four of 256 threads, of which three find
// room for 64 KB, eight of 128 with parts of at most 32 KB, or 16 of 64: what
// a small part costs is the latency of its steps, and more of them overlap.
template <int NT>
constexpr int kBlocks = 1024 / NT;
constexpr int kSmallPart = 32 * 1024, kTinyPart = 8 * 1024;

// What the blocks of a cluster tell each other about a row: the part's
// maximum and sum, and of the kept tokens in it the sums of
// w (x - m) and of w, with w_j = kShare 2^((teacher_j - max) c).
struct Share {
  float m, s, gap, w;
};

struct RowShared {
  Share of_block[kMaxCluster], careful[kMaxCluster];
  float m[kMaxWarps], tmax[kMaxWarps], s[kMaxWarps], gap[kMaxWarps], w[kMaxWarps], z[kMaxWarps], own[kMaxWarps];
  float single[32];
};

template <int NW>
__device__ __forceinline__ float sum_of(const float* v) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) s += v[i];
  return s;
}
template <int NW>
__device__ __forceinline__ float max_of_warps(const float* v) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) m = max_nan(m, v[i]);
  return m;
}

// A row as the gradient needs it.
struct Joined {
  float ref, l2s;  // log2 q_v = (x_v - ref) c - l2s
  float gap;       // sum w (x - ref) over the kept tokens
  bool empty;      // every logit is masked
  bool fast;       // the fast statistic holds
};

template <typename T, int NT, int G>
__device__ __forceinline__ void take_group(Run& run, int nvec, uint32_t mine, float c) {
  cp_async_wait<kGroups - 1 - G>();
  const int first = (int)threadIdx.x + G * kUnroll * NT;
  const uint32_t from = mine + G * kUnroll * NT * 16;
  if (first + (kUnroll - 1) * NT < nvec) {
    uint4 r[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) r[k] = ld_shared_v4(from + k * NT * 16);
    add_vectors<T, false>(run, r, max_of<T>(r), c);
  } else {
#pragma unroll 1
    for (int k = 0; first + k * NT < nvec; ++k) {
      const uint4 r[1] = {ld_shared_v4(from + k * NT * 16)};
      add_vectors<T, false>(run, r, max_of<T>(r), c);
    }
  }
  if constexpr (G + 1 < kGroups) take_group<T, NT, G + 1>(run, nvec, mine, c);
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, kBlocks<NT>) distill_grad_kernel(RowArgs a, int C, int room) {
  constexpr int V = kVec<T>, NW = NT / 32;
  extern __shared__ __align__(16) unsigned char raw[];  // [room] vectors, then the kept slots
  __shared__ RowShared sh;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = C == 1 ? 0 : (int)(blockIdx.x % C);
  const long long row = blockIdx.x / C;
  const int len = part_len(a.V, C);
  const int lo = (int)min((long long)a.V, (long long)rank * len), hi = (int)min((long long)a.V, (long long)lo + len);
  const float c = kLog2e / a.temperature;
  cg::cluster_group cl = cg::this_cluster();
  const T* xr = static_cast<const T*>(a.x) + row * a.x_stride;
  const Part<T> p(xr, lo, hi);
  const T* part = reinterpret_cast<const T*>(raw);  // from p.vec(0) on
  const uint32_t mine = smem_u32(raw) + t * 16;     // this thread's first vector
  int* id = reinterpret_cast<int*>(raw + (size_t)room * 16);  // kept token, or -1
  float* w = reinterpret_cast<float*>(id + a.K);              // teacher's value, then kShare 2^((value - max) c)
  float* x = w + a.K;                                         // the student's logit, by the thread that has the slot

  // everything the row needs is on its way at once
  for (int j = t; j < a.K; j += NT) {
    cp_async4(smem_u32(id + j), a.ids + row * a.K + j);
    cp_async4(smem_u32(w + j), a.teacher + row * a.K + j);
  }
  cp_async_commit();
  const T* from = p.vec(t);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int o = (g * kUnroll + k) * NT;
      if (t + o < p.nvec) cp_async16(mine + o * 16, from + o * V, 16);
    }
    cp_async_commit();
  }
  T one = from_f32<T>(0.f);
  if (t < p.singles()) one = p.head[p.single_at(t)];
  float g = a.temperature * a.grad_scale;
  if (a.dloss) g *= a.dloss[row];
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // every block has started

  Run run{kFloor, {0.f, 0.f}, {0.f, 0.f}};
  take_group<T, NT, 0>(run, p.nvec, mine, c);
  if (t < p.singles()) {
    const float v = to_f32(one);
    raise(run, fmaxf(v, kFloor), c, false);
    run.s.x += ex2((floor_nan(v) - run.m) * c);
    sh.single[t] = v;
  }
  prefetch_part<T>(a, row, lo, hi, kRoom<NT> * 16);
  float tmax = NEG_INF;
  for (int j = t; j < a.K; j += NT) {
    if (id[j] >= 0 && id[j] < a.V) {
      tmax = max_nan(tmax, w[j]);
    } else {
      id[j] = -1;
      w[j] = NEG_INF;
    }
  }
  const float wm = warp_max_f(run.m);
  tmax = warp_max_f(tmax);
  if (lane == 0) {
    sh.m[warp] = wm;
    sh.tmax[warp] = tmax;
  }
  __syncthreads();  // also: every thread's copies and single elements are there
  Stat own{run.m, run.s.x + run.s.y, 0.f};
  const float m = max_of_warps<NW>(sh.m);
  tmax = max_of_warps<NW>(sh.tmax);
  const float tref = finite_max(tmax);
  rescale(own, m, c);
  // of the teacher's slots: z = sum w, sum w (teacher - max); of those in this
  // part sum w (x - m) and sum w
  float z = 0.f, w_log_w = 0.f, gap = 0.f, here = 0.f;
  if (warp * 32 < a.K) {
    for (int j = t; j < a.K; j += NT) {
      const float d = w[j] - tref, wj = ex2(d * c) * kShare;
      w[j] = wj;
      z += wj;
      // in the logits' units: a lowest-value mask stays finite there
      if (wj > 0.f) w_log_w += wj * d;
      if (id[j] >= lo && id[j] < hi) {
        const int e = id[j] - lo - p.nhead;
        float xj;
        if (e < 0)
          xj = sh.single[e + p.nhead];
        else if (e >= p.nvec * V)
          xj = sh.single[p.nhead + e - p.nvec * V];
        else
          xj = to_f32(part[e]);
        x[j] = xj;
        if (wj > 0.f) gap += wj * (xj - m);
        here += wj;
      }
    }
    z = warp_sum(z);
    w_log_w = warp_sum(w_log_w);
    gap = warp_sum(gap);
    here = warp_sum(here);
  }
  own.s = warp_sum(own.s);
  if (lane == 0) {
    sh.s[warp] = own.s;
    sh.z[warp] = z;
    sh.own[warp] = w_log_w;
    sh.gap[warp] = gap;
    sh.w[warp] = here;
  }
  __syncthreads();
  z = sum_of<NW>(sh.z);
  if (C > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (t < C) *cl.map_shared_rank(&sh.of_block[rank], t) = Share{m, sum_of<NW>(sh.s), sum_of<NW>(sh.gap), sum_of<NW>(sh.w)};
    cl.sync();
  } else {
    if (t == 0) sh.of_block[0] = Share{m, sum_of<NW>(sh.s), sum_of<NW>(sh.gap), sum_of<NW>(sh.w)};
    __syncthreads();
  }

  auto join = [&](const Share* of) {
    float top = of[0].m;
    for (int i = 1; i < C; ++i) top = fmaxf(top, of[i].m);
    Joined r;
    r.ref = finite_max(top);
    float s = 0.f;
    r.gap = 0.f;
    for (int i = 0; i < C; ++i) {
      Stat o{of[i].m, of[i].s, 0.f};
      rescale(o, top, c);
      s += o.s;
      if (of[i].w > 0.f) r.gap += of[i].gap + of[i].w * (of[i].m - r.ref);
    }
    r.empty = top == NEG_INF && s == 0.f;  // (s is NaN where the row holds a NaN)
    r.l2s = log2f(s);
    r.fast = top > kFloor && c >= kLeastScale && c <= kMostScale;
    return r;
  };
  Joined r = join(sh.of_block);
  if (!r.fast) {  // uniform over the cluster: a row that the fast statistic does not hold for
    Stat any = part_stat_any<NT, T, false>(p, c);
    const float wm2 = warp_max_f(any.m);
    __syncthreads();
    if (lane == 0) sh.m[warp] = wm2;
    __syncthreads();
    const float m2 = max_of_warps<NW>(sh.m);
    rescale(any, m2, c);
    any.s = warp_sum(any.s);
    if (lane == 0) sh.s[warp] = any.s;
    __syncthreads();
    if (C > 1) {
      if (t < C) *cl.map_shared_rank(&sh.careful[rank], t) = Share{m2, sum_of<NW>(sh.s), 0.f, 0.f};
      cl.sync();
    } else {
      if (t == 0) sh.careful[0] = Share{m2, sum_of<NW>(sh.s), 0.f, 0.f};
      __syncthreads();
    }
    r = join(sh.careful);
    gap = 0.f;
    for (int j = t; j < a.K; j += NT)
      if (w[j] > 0.f) gap += w[j] * (to_f32(xr[id[j]]) - r.ref);
    gap = warp_sum(gap);
    if (lane == 0) sh.gap[warp] = gap;
    __syncthreads();
    r.gap = sum_of<NW>(sh.gap);
    if (C > 1) cl.sync();  // before any block writes its gradient over the logits
  }

  const bool zero = tmax == NEG_INF || r.empty;
  if (rank == 0 && t == 0 && a.loss)
    a.loss[row] =
        zero ? 0.f : loss_of((sum_of<NW>(sh.own) - r.gap) / z, r.l2s - log2f(z / kShare), a.temperature);
  T* dst = static_cast<T*>(a.dx) + row * a.dx_stride + lo;
  if (zero) {
    for (int i = t; i < hi - lo; i += NT) dst[i] = from_f32<T>(0.f);
    return;
  }
  const float2 c2 = both(c), nref = both(-r.ref), off = both(-r.l2s), g2 = both(g);
  auto grad = [&](float2 v) {
    const float2 d = fma2(add2(v, nref), c2, off);
    return mul2(make_float2(ex2(d.x), ex2(d.y)), g2);
  };
  if (((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(p.head)) & 15) == 0) {
    T* dv = dst + p.nhead;
    int i = t;
    uint32_t at = mine;
    for (; i + (kUnroll - 1) * NT < p.nvec; i += kUnroll * NT, at += kUnroll * NT * 16) {
      uint4 v[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) v[k] = ld_shared_v4(at + k * NT * 16);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) st_stream(dv + (long long)(i + k * NT) * V, map_vector<T>(v[k], grad));
    }
    for (; i < p.nvec; i += NT, at += NT * 16)
      st_stream(dv + (long long)i * V, map_vector<T>(ld_shared_v4(at), grad));
  } else {
#pragma unroll 4
    for (int i = t; i < p.nvec * V; i += NT) dst[p.nhead + i] = from_f32<T>(grad(both(to_f32(part[i]))).x);
  }
  if (t < p.singles()) dst[p.single_at(t)] = from_f32<T>(grad(both(sh.single[t])).x);
  __syncthreads();
  // the kept tokens of this part, once each
  const float iz = 1.f / z;
  for (int j = t; j < a.K; j += NT) {
    if (id[j] < lo || id[j] >= hi) continue;
    float pj = 0.f;
    bool first = true;
#pragma unroll 4
    for (int k = 0; k < a.K; ++k)
      if (id[k] == id[j]) {
        if (k < j) first = false;
        pj += w[k];
      }
    if (first) dst[id[j] - lo] = from_f32<T>(grad(both(x[j])).x - g * pj * iz);
  }
}

// Blocks a row (0: it is too wide): as few as hold it, and more where few
// rows would leave SMs idle.
int blocks_of(const RowArgs& a) {
  const int vec = a.type == 0 ? 4 : 8;
  int C = 1;
  while (C < kMaxCluster && a.rows * 2 * C <= a.num_sms && a.V >= 8LL * C * 256 * vec) C *= 2;
  while (C <= kMaxCluster && part_len(a.V, C) / vec > kRoom<256>) C *= 2;
  return C <= kMaxCluster ? C : 0;
}

template <typename T, int NT>
cudaError_t launch_parts(RowArgs a, int C, cudaStream_t st) {
  const int room = part_len(a.V, C) / kVec<T>;
  const size_t smem = (size_t)room * 16 + a.K * 12;
  const auto kern = distill_grad_kernel<T, NT>;
  static std::atomic<size_t> limit[64];
  const cudaError_t e = raise_smem((const void*)kern, (size_t)kRoom<NT> * 16 + IBWD_MAX_KEPT * 12, limit);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  a.ahead = std::max(1, 2 * a.num_sms / C);  // (two or three blocks an SM: 368 and 370 us)
  cfg.gridDim = dim3((unsigned)(a.rows * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, C, room);
}

template <typename T>
cudaError_t launch_typed(const RowArgs& a, cudaStream_t st) {
  const int C = blocks_of(a);
  const int bytes = part_len(a.V, C) * (int)sizeof(T);
  if (a.rows * C <= 2 * a.num_sms) return launch_parts<T, 256>(a, C, st);
  if (bytes <= kTinyPart) return launch_parts<T, 64>(a, C, st);
  return bytes <= kSmallPart ? launch_parts<T, 128>(a, C, st) : launch_parts<T, 256>(a, C, st);
}

}  // namespace

bool distill_resident(const RowArgs& a) { return blocks_of(a) != 0; }

cudaError_t launch_distill_resident(const RowArgs& a, cudaStream_t st) {
  switch (a.type) {
    case 0: return launch_typed<float>(a, st);
    case 1: return launch_typed<__nv_bfloat16>(a, st);
    default: return launch_typed<__half>(a, st);
  }
}

}  // namespace ibwd
