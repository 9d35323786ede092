// Layer norm over the rows of a matrix, forward and backward, on sm_103a:
//   y = (x - mean) rstd gamma + beta,
//   dx = rstd (d - sum(d)/N - xh sum(d xh)/N),  xh = (x - mean) rstd, d = dy gamma,
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy.
#include <algorithm>

#include "elem.cuh"
#include "kcommon.cuh"
#include "train.h"

namespace ibwd {
namespace {

constexpr int kThreads = 256;

// gamma / beta element n as fp32: fp32 or the type of x.
template <typename T>
__device__ __forceinline__ float weight(const void* w, int n, bool f32, float none) {
  if (w == nullptr) return none;
  return f32 ? static_cast<const float*>(w)[n] : to_f32(static_cast<const T*>(w)[n]);
}

// Sums of K values over the block, the same bits in every thread.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float* stage) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  __syncthreads();
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) stage[warp * K + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < nw; ++w)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += stage[w * K + k];
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads) norm_fwd_any(NormFwdArgs a) {
  __shared__ float stage[32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const TX* x = static_cast<const TX*>(a.x) + r * a.x_stride;
    TY* y = static_cast<TY*>(a.y) + r * a.y_stride;
    float s[1] = {0.f};
    for (int n = threadIdx.x; n < a.N; n += kThreads) s[0] += to_f32(x[n]);
    block_sums(s, stage);
    const float mean = s[0] / a.N;
    float q[1] = {0.f};
    for (int n = threadIdx.x; n < a.N; n += kThreads) {
      const float d = to_f32(x[n]) - mean;
      q[0] += d * d;
    }
    block_sums(q, stage);
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
__global__ void __launch_bounds__(kThreads) norm_bwd_rows_any(NormBwdArgs a) {
  __shared__ float stage[64];
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
    block_sums(s, stage);
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
__global__ void __launch_bounds__(kThreads) norm_bwd_columns_any(NormBwdArgs a, int group_rows) {
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

// dgamma and dbeta from the groups' column sums, in the groups' order.
__global__ void __launch_bounds__(kThreads) norm_bwd_join(const float* part, int groups, int N, float* dgamma,
                                                          float* dbeta) {
  const int n = blockIdx.x * kThreads + threadIdx.x;
  if (n >= N) return;
  float g = 0.f, b = 0.f;
  for (int i = 0; i < groups; ++i) {
    g += part[(2LL * i) * N + n];
    b += part[(2LL * i + 1) * N + n];
  }
  if (dgamma) dgamma[n] = g;
  if (dbeta) dbeta[n] = b;
}

constexpr int kMaxGroups = 64;

int groups_of(long long rows) { return (int)std::min<long long>(kMaxGroups, std::max<long long>(1, (rows + 31) / 32)); }

template <typename TX, typename TD>
cudaError_t bwd_any(const NormBwdArgs& a, cudaStream_t st) {
  if (a.dgamma || a.dbeta) {  // first: dx may be x or dy
    const int groups = groups_of(a.rows);
    const int group_rows = (int)((a.rows + groups - 1) / groups);
    norm_bwd_columns_any<TX, TD><<<dim3((a.N + 31) / 32, groups), kThreads, 0, st>>>(a, group_rows);
    norm_bwd_join<<<(a.N + kThreads - 1) / kThreads, kThreads, 0, st>>>(a.part, groups, a.N, a.dgamma, a.dbeta);
  }
  const int grid = (int)std::min<long long>(a.rows, 8LL * a.num_sms);
  if (grid) norm_bwd_rows_any<TX, TD><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t fwd_any(const NormFwdArgs& a, cudaStream_t st) {
  if (!a.rows) return cudaSuccess;
  norm_fwd_any<TX, TY><<<(int)std::min<long long>(a.rows, 8LL * a.num_sms), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_workspace(long long rows, int N) { return (size_t)groups_of(rows) * 2 * N * sizeof(float); }

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.x_type == 0) {
    if (a.y_type == 0) return fwd_any<float, float>(a, st);
    if (a.y_type == 1) return fwd_any<float, bf>(a, st);
    return fwd_any<float, __half>(a, st);
  }
  return a.x_type == 1 ? fwd_any<bf, bf>(a, st) : fwd_any<__half, __half>(a, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.x_type == 0) {
    if (a.dy_type == 0) return bwd_any<float, float>(a, st);
    if (a.dy_type == 1) return bwd_any<float, bf>(a, st);
    return bwd_any<float, __half>(a, st);
  }
  if (a.x_type == 1) return a.dy_type == 0 ? bwd_any<bf, float>(a, st) : bwd_any<bf, bf>(a, st);
  return a.dy_type == 0 ? bwd_any<__half, float>(a, st) : bwd_any<__half, __half>(a, st);
}

}  // namespace ibwd
