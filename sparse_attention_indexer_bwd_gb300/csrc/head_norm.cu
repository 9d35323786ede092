// Norm and rotation of queries and keys: the launch by type, and the join of
// the backward pass's column sums.
#include "head_norm.cuh"

namespace ibwd {

namespace {

// A thread column for 32 of the D columns, 32 slices of the blocks each; the
// slices meet in shared memory in a fixed order.
__global__ void __launch_bounds__(1024) join_kernel(const __grid_constant__ HeadArgs a) {
  __shared__ float sum[32][33];
  const HeadOp& o = a.op[blockIdx.z];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, first = blockIdx.z ? a.op[0].blocks : 0;
  float* to = blockIdx.y ? o.dbeta : o.dgamma;
  chained();
  float v = 0.f;
  const bool on = col < a.D && to && o.norm != IBWD_NORM_NONE;
  if (on) {
    const float* p = a.part + blockIdx.y * (long long)a.D + col;
#pragma unroll 4
    for (int b = slice; b < o.blocks; b += 32) v += p[(long long)(first + b) * 2 * a.D];
  }
  sum[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && on) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sum[i][lane];
    to[col] = s;
  }
}

}  // namespace

cudaError_t join_heads(const HeadArgs& a, cudaStream_t st) {
  bool any = false;
  for (const HeadOp& o : a.op) any = any || (o.norm != IBWD_NORM_NONE && (o.dgamma || o.dbeta));
  if (!any) return cudaSuccess;
  return launch_ex(join_kernel, dim3((a.D + 31) / 32, 2, 2), 1024u, 0, st, true, a);
}

cudaError_t launch_heads(const HeadArgs& a, bool backward, cudaStream_t st) {
  if (a.type == IBWD_F32) return heads_f32(a, backward, st);
  if (a.type == IBWD_BF16) return heads_bf16(a, backward, st);
  return heads_f16(a, backward, st);
}

}  // namespace ibwd
