// Layer norm over the rows of a matrix, forward and backward, on sm_103a:
//   y = (x - mean) rstd gamma + beta,
//   dx = rstd (d - sum(d)/N - xh sum(d xh)/N),  xh = (x - mean) rstd, d = dy gamma,
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy.
// About ten operations an element beside four to twelve bytes: bound by HBM,
// or by the launch where rows are few.
//
// A team of threads holds a row in registers (16 elements a thread at most),
// so every element is read once: 8 to 32 lanes of a warp for short rows, a
// thread block for longer ones.  Teams stay resident and walk the rows, the
// next row's loads in flight while the current one is reduced; gamma and beta
// stay in registers, and so do the backward pass's column sums of the team's
// rows.  Those meet in a fixed order: a block's teams in shared memory, the
// blocks of a cluster through distributed shared memory, the clusters in a
// second small kernel.  Rows too wide for a block take several passes.
#include <cooperative_groups.h>

#include <algorithm>

#include "elem.cuh"
#include "kcommon.cuh"
#include "train.h"

namespace cg = cooperative_groups;

namespace ibwd {
namespace {

constexpr int kThreads = 256;     // block of several teams, and of the kernels for wide rows
constexpr int kMaxTeam = 512;     // threads of a block that is one team
constexpr int kCluster = 8;       // blocks whose column sums meet before they are written
constexpr int kElems = 16;        // elements of a row a thread holds at most
constexpr int kMaxTeamWidth = kMaxTeam * kElems;

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
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = e[i];
    }
  }
};

// gamma / beta element n as fp32: fp32 or the type of x.
template <typename T>
__device__ __forceinline__ float weight(const void* w, int n, bool f32, float none) {
  if (w == nullptr) return none;
  return f32 ? static_cast<const float*>(w)[n] : to_f32(static_cast<const T*>(w)[n]);
}

// Sums of K values over a team, the same bits in each of its threads.  TEAM
// lanes of a warp, or 0 for the block: then `stage` holds 2 * 32 * K floats,
// used in turn (`turn` flips), so one barrier a call is enough.
template <int TEAM, int K>
__device__ __forceinline__ void team_sums(float (&v)[K], float* stage, int& turn) {
#pragma unroll
  for (int o = (TEAM ? TEAM : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (TEAM == 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    float* s = stage + turn * 32 * K;
    turn ^= 1;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[warp * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int w = 0; w < nw; ++w)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += s[w * K + k];
  }
}

template <typename TX, typename TY, int VEC, int K, int TEAM>
__global__ void __launch_bounds__(TEAM ? kThreads : kMaxTeam) norm_fwd_team(NormFwdArgs a) {
  __shared__ float stage[64];
  constexpr int TPB = TEAM ? kThreads / (TEAM ? TEAM : 1) : 1;
  const int team = TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0;
  const int t = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x, T = TEAM ? TEAM : blockDim.x;
  const int nvec = a.N / VEC;
  const float inv_n = 1.f / a.N;
  float g[K][VEC], b[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int j = t + k * T, n = j * VEC + i;
      g[k][i] = j < nvec ? weight<TX>(a.gamma, n, a.w_type == 0, 1.f) : 0.f;
      b[k][i] = j < nvec ? weight<TX>(a.beta, n, a.w_type == 0, 0.f) : 0.f;
    }
  Chunk<TX, VEC> cur[K], nxt[K];
  auto load = [&](Chunk<TX, VEC>(&c)[K], long long r) {
    const TX* x = static_cast<const TX*>(a.x) + r * a.x_stride;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (r < a.rows && t + k * T < nvec) c[k].load(x + (t + k * T) * VEC);
  };
  int turn = 0;
  const long long step = (long long)gridDim.x * TPB;
  long long base = (long long)blockIdx.x * TPB;
  load(cur, base + team);
  for (; base < a.rows; base += step) {
    const long long r = base + team;
    load(nxt, r + step);
    float v[K][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[k][i] = t + k * T < nvec ? to_f32(cur[k].e[i]) : 0.f;
        s[0] += v[k][i];
      }
    team_sums<TEAM>(s, stage, turn);
    const float mean = s[0] / a.N;  // (a constant row has its mean exactly)
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t + k * T < nvec)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          v[k][i] -= mean;
          q[0] = fmaf(v[k][i], v[k][i], q[0]);
        }
    team_sums<TEAM>(q, stage, turn);
    const float rstd = 1.f / sqrtf(fmaf(q[0], inv_n, a.eps));
    if (r < a.rows) {
      TY* y = static_cast<TY*>(a.y) + r * a.y_stride;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k * T < nvec) {
          Chunk<TY, VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) o.e[i] = from_f32<TY>(fmaf(v[k][i] * rstd, g[k][i], b[k][i]));
          o.store(y + (t + k * T) * VEC);
        }
      if (t == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) cur[k] = nxt[k];
  }
}

// Column sums of a block, [2][N] in shared memory in the order of the
// teams, written to part[group] -- or, where there is only one group, to
// dgamma and dbeta.  A cluster's blocks first add up: each takes a share of
// the columns over the blocks in their order.
__device__ __forceinline__ void write_sums(const NormBwdArgs& a, const float* sums, int cluster) {
  const int n2 = 2 * a.N;
  const int groups = gridDim.x / cluster, group = blockIdx.x / cluster;
  auto put = [&](int c, float v) {
    if (groups > 1)
      a.part[(long long)group * n2 + c] = v;
    else if (c < a.N) {
      if (a.dgamma) a.dgamma[c] = v;
    } else if (a.dbeta)
      a.dbeta[c - a.N] = v;
  };
  if (cluster == 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < n2; c += blockDim.x) put(c, sums[c]);
    return;
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  const int rank = (int)cl.block_rank();
  for (int c = rank * blockDim.x + threadIdx.x; c < n2; c += kCluster * blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kCluster; ++i) v += *cl.map_shared_rank(sums + c, i);
    put(c, v);
  }
  cl.sync();  // no block leaves while its sums are read
}

template <typename TX, typename TD, int VEC, int K, int TEAM>
__global__ void __launch_bounds__(TEAM ? kThreads : kMaxTeam) norm_bwd_team(NormBwdArgs a, int cluster) {
  extern __shared__ float sums[];  // [2][N]
  __shared__ float stage[128];
  constexpr int TPB = TEAM ? kThreads / (TEAM ? TEAM : 1) : 1;
  // single elements take a register each: 16 of two rows would spill
  constexpr bool kAhead = VEC > 1;
  const int team = TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0;
  const int t = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x, T = TEAM ? TEAM : blockDim.x;
  const int nvec = a.N / VEC;
  const float inv_n = 1.f / a.N;
  float g[K][VEC], dg[K][VEC], db[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int j = t + k * T;
      g[k][i] = j < nvec ? weight<TX>(a.gamma, j * VEC + i, a.w_type == 0, 1.f) : 0.f;
      dg[k][i] = db[k][i] = 0.f;
    }
  Chunk<TX, VEC> cx[K], nx[K];
  Chunk<TD, VEC> cd[K], nd[K];
  float cm = 0.f, cr = 0.f, nm = 0.f, nr = 0.f;
  auto load = [&](Chunk<TX, VEC>(&x)[K], Chunk<TD, VEC>(&d)[K], float& mean, float& rstd, long long r) {
    if (r >= a.rows) return;
    const TX* px = static_cast<const TX*>(a.x) + r * a.x_stride;
    const TD* pd = static_cast<const TD*>(a.dy) + r * a.dy_stride;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (t + k * T < nvec) {
        x[k].load(px + (t + k * T) * VEC);
        d[k].load(pd + (t + k * T) * VEC);
      }
    mean = a.mean[r];
    rstd = a.rstd[r];
  };
  int turn = 0;
  const long long step = (long long)gridDim.x * TPB;
  long long base = (long long)blockIdx.x * TPB;
  if (kAhead) load(cx, cd, cm, cr, base + team);
  for (; base < a.rows; base += step) {
    const long long r = base + team;
    const bool on = r < a.rows;
    if (kAhead)
      load(nx, nd, nm, nr, r + step);
    else
      load(cx, cd, cm, cr, r);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (on && t + k * T < nvec)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xh = (to_f32(cx[k].e[i]) - cm) * cr, dy = to_f32(cd[k].e[i]);
          const float d = dy * g[k][i];
          dg[k][i] = fmaf(dy, xh, dg[k][i]);
          db[k][i] += dy;
          s[0] += d;
          s[1] = fmaf(d, xh, s[1]);
        }
    team_sums<TEAM>(s, stage, turn);
    if (on) {
      const float ma = s[0] * inv_n, mb = s[1] * inv_n;
      TX* dx = static_cast<TX*>(a.dx) + r * a.dx_stride;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k * T < nvec) {
          Chunk<TX, VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float xh = (to_f32(cx[k].e[i]) - cm) * cr;
            o.e[i] = from_f32<TX>(cr * (fmaf(to_f32(cd[k].e[i]), g[k][i], -ma) - xh * mb));
          }
          o.store(dx + (t + k * T) * VEC);
        }
    }
    if (kAhead) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        cx[k] = nx[k];
        cd[k] = nd[k];
      }
      cm = nm;
      cr = nr;
    }
  }
  if (!a.dgamma && !a.dbeta) return;
  // the teams' sums, in the teams' order
  for (int w = 0; w < TPB; ++w) {
    if (w == team)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k * T < nvec)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int c = (t + k * T) * VEC + i;
            sums[c] = w ? sums[c] + dg[k][i] : dg[k][i];
            sums[a.N + c] = w ? sums[a.N + c] + db[k][i] : db[k][i];
          }
    if (TPB > 1) __syncthreads();
  }
  griddep_launch_dependents();
  write_sums(a, sums, cluster);
}

// dgamma and dbeta from the groups' column sums [groups][2][N]: 32 columns a
// block, eight interleaved sums of groups each, joined in order.
__global__ void __launch_bounds__(kThreads) norm_bwd_join(const float* part, int groups, int N, float* dgamma,
                                                          float* dbeta) {
  __shared__ float s[8][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < 2 * N) {
#pragma unroll 4
    for (int i = w; i < groups; i += 8) v += part[(long long)i * 2 * N + c];
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < 2 * N) {
    v = 0.f;
    for (int i = 0; i < 8; ++i) v += s[i][lane];
    if (c < N) {
      if (dgamma) dgamma[c] = v;
    } else if (dbeta)
      dbeta[c - N] = v;
  }
}

// ------------------------------------------------------------- wide rows ---
// Any width and alignment: a block takes a row in three passes (two backward).

template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads) norm_fwd_wide(NormFwdArgs a) {
  __shared__ float stage[64];
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
  __shared__ float stage[128];
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
    a.part[((long long)blockIdx.y * 2) * a.N + n] = g;
    a.part[((long long)blockIdx.y * 2 + 1) * a.N + n] = b;
  }
}

// -------------------------------------------------------------- launches ---

constexpr int kMaxSms = 160;       // the workspace does not depend on the device
constexpr int kMaxWideGroups = 64;

// The shape of a team launch: threads of the block, blocks, cluster.
struct TeamShape {
  int threads, blocks, cluster;
};

// teams_per_block 0: the block is the team.  About `per_sm` threads an SM.
TeamShape team_shape(long long rows, int N, int elems, int teams_per_block, int per_sm, int num_sms, bool sums) {
  TeamShape s;
  if (teams_per_block) {
    s.threads = kThreads;
    s.blocks = (int)std::min<long long>((rows + teams_per_block - 1) / teams_per_block,
                                        (long long)num_sms * (per_sm / kThreads));
    s.cluster = 1;
    return s;
  }
  s.threads = std::max(32, ((N + elems - 1) / elems + 31) / 32 * 32);
  s.blocks = (int)std::min<long long>(rows, (long long)num_sms * std::max(1, per_sm / s.threads));
  s.cluster = 1;
  if (sums) {
    // column sums meet in clusters; up to 16 rows one cluster takes them all
    // and writes the results itself
    s.cluster = kCluster;
    s.blocks = rows <= 2 * kCluster ? kCluster : (s.blocks + kCluster - 1) / kCluster * kCluster;
  }
  return s;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), const TeamShape& s, size_t smem, cudaStream_t st, Args... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(s.blocks);
  cfg.blockDim = dim3(s.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = s.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = s.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

bool aligned(const void* p, long long stride, int size, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * size % bytes == 0;
}

constexpr int kFwdPerSm = 768, kBwdPerSm = 512;

template <typename TX, typename TY, int VEC, int K, int TEAM>
cudaError_t fwd_team(const NormFwdArgs& a, cudaStream_t st) {
  const TeamShape s = team_shape(a.rows, a.N, VEC * K, TEAM ? kThreads / (TEAM ? TEAM : 1) : 0, kFwdPerSm, a.num_sms,
                                 false);
  return launch_cluster(norm_fwd_team<TX, TY, VEC, K, TEAM>, s, 0, st, a);
}

template <typename TX, typename TY>
cudaError_t norm_fwd(const NormFwdArgs& a, cudaStream_t st) {
  constexpr int V = kVec<TX>;
  const int ysize = (int)sizeof(TY);
  if (a.N > kMaxTeamWidth) {
    norm_fwd_wide<TX, TY><<<(int)std::min<long long>(a.rows, 8LL * a.num_sms), kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  // whole 16-byte vectors of x where every row allows it, else elements
  if (a.N % V == 0 && aligned(a.x, a.x_stride, sizeof(TX), 16) && aligned(a.y, a.y_stride, ysize, V * ysize)) {
    if (a.N <= 8 * V) return fwd_team<TX, TY, V, 1, 8>(a, st);
    if (a.N <= 16 * V) return fwd_team<TX, TY, V, 1, 16>(a, st);
    if (a.N <= 32 * V) return fwd_team<TX, TY, V, 1, 32>(a, st);
    if (a.N <= 32 * kElems) return fwd_team<TX, TY, V, kElems / V, 32>(a, st);
    return fwd_team<TX, TY, V, kElems / V, 0>(a, st);
  }
  if (a.N <= 128) return fwd_team<TX, TY, 1, 4, 32>(a, st);
  if (a.N <= 32 * kElems) return fwd_team<TX, TY, 1, kElems, 32>(a, st);
  return fwd_team<TX, TY, 1, kElems, 0>(a, st);
}

cudaError_t join_sums(const NormBwdArgs& a, int groups, cudaStream_t st) {
  return launch_ex(norm_bwd_join, (2 * a.N + 31) / 32, kThreads, 0, st, true, (const float*)a.part, groups, a.N,
                   a.dgamma, a.dbeta);
}

template <typename TX, typename TD, int VEC, int K, int TEAM>
cudaError_t bwd_team(const NormBwdArgs& a, cudaStream_t st) {
  const bool sums = a.dgamma || a.dbeta;
  const TeamShape s = team_shape(a.rows, a.N, VEC * K, TEAM ? kThreads / (TEAM ? TEAM : 1) : 0, kBwdPerSm, a.num_sms,
                                 sums);
  cudaError_t e = launch_cluster(norm_bwd_team<TX, TD, VEC, K, TEAM>, s, sums ? 2 * a.N * sizeof(float) : 0, st, a,
                                 s.cluster);
  const int groups = s.blocks / s.cluster;
  if (e == cudaSuccess && sums && groups > 1) e = join_sums(a, groups, st);
  return e;
}

template <typename TX, typename TD>
cudaError_t norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  constexpr int V = kVec<TX>;
  const int dsize = (int)sizeof(TD);
  const bool sums = a.dgamma || a.dbeta;
  if (!a.rows) {
    if (a.dgamma) cudaMemsetAsync(a.dgamma, 0, a.N * sizeof(float), st);
    if (a.dbeta) cudaMemsetAsync(a.dbeta, 0, a.N * sizeof(float), st);
    return cudaGetLastError();
  }
  if (a.N > kMaxTeamWidth) {
    if (sums) {  // before the rows: dx may be x or dy
      const int groups = (int)std::min<long long>(kMaxWideGroups, (a.rows + 31) / 32);
      const int group_rows = (int)((a.rows + groups - 1) / groups);
      norm_bwd_wide_columns<TX, TD><<<dim3((a.N + 31) / 32, groups), kThreads, 0, st>>>(a, group_rows);
      cudaError_t e = cudaGetLastError();
      if (e == cudaSuccess) e = join_sums(a, groups, st);
      if (e != cudaSuccess) return e;
    }
    norm_bwd_wide<TX, TD><<<(int)std::min<long long>(a.rows, 8LL * a.num_sms), kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  if (a.N % V == 0 && aligned(a.x, a.x_stride, sizeof(TX), 16) && aligned(a.dx, a.dx_stride, sizeof(TX), 16) &&
      aligned(a.dy, a.dy_stride, dsize, std::min(16, V * dsize))) {
    if (a.N <= 8 * V) return bwd_team<TX, TD, V, 1, 8>(a, st);
    if (a.N <= 16 * V) return bwd_team<TX, TD, V, 1, 16>(a, st);
    if (a.N <= 32 * V) return bwd_team<TX, TD, V, 1, 32>(a, st);
    if (a.N <= 32 * kElems) return bwd_team<TX, TD, V, kElems / V, 32>(a, st);
    return bwd_team<TX, TD, V, kElems / V, 0>(a, st);
  }
  if (a.N <= 128) return bwd_team<TX, TD, 1, 4, 32>(a, st);
  if (a.N <= 32 * kElems) return bwd_team<TX, TD, 1, kElems, 32>(a, st);
  return bwd_team<TX, TD, 1, kElems, 0>(a, st);
}

}  // namespace

// Column sums of every group any launch for this shape makes: a block of
// several teams is a group of its own, eight blocks of one team are one.
size_t norm_bwd_workspace(long long rows, int N) {
  long long groups = kMaxWideGroups;
  if (N <= 32 * kElems)
    groups = std::min<long long>((rows + 7) / 8, (long long)kMaxSms * (kBwdPerSm / kThreads));
  else if (N <= kMaxTeamWidth)
    groups = (std::min<long long>(rows, (long long)kMaxSms * (kBwdPerSm / 32)) + kCluster - 1) / kCluster;
  else
    groups = std::min<long long>(kMaxWideGroups, (rows + 31) / 32);
  return (size_t)std::max<long long>(1, groups) * 2 * N * sizeof(float);
}

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.x_type == 0) {
    if (a.y_type == 0) return norm_fwd<float, float>(a, st);
    if (a.y_type == 1) return norm_fwd<float, bf>(a, st);
    return norm_fwd<float, __half>(a, st);
  }
  return a.x_type == 1 ? norm_fwd<bf, bf>(a, st) : norm_fwd<__half, __half>(a, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.x_type == 0) {
    if (a.dy_type == 0) return norm_bwd<float, float>(a, st);
    if (a.dy_type == 1) return norm_bwd<float, bf>(a, st);
    return norm_bwd<float, __half>(a, st);
  }
  if (a.x_type == 1) return a.dy_type == 0 ? norm_bwd<bf, float>(a, st) : norm_bwd<bf, bf>(a, st);
  return a.dy_type == 0 ? norm_bwd<__half, float>(a, st) : norm_bwd<__half, __half>(a, st);
}

}  // namespace ibwd
