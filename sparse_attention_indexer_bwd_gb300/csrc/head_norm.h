// Launchers of the norm and rotation of queries and keys (head_norm.cuh),
// shared by head_norm.cu and one translation unit a type of the heads.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ibwd {

// One operand: the heads of the queries, or those of the keys.
struct HeadOp {
  const void* x;
  const void* dy;  // backward
  void* y;         // the result, dx in the backward pass
  const void* gamma;
  const void* beta;
  float* dgamma;  // or nullptr
  float* dbeta;
  long long x_token, x_head, dy_token, dy_head, y_token, y_head;  // strides in elements
  int heads;                                                      // 0: absent
  int norm;                                                       // ibwd_norm
  int dy_f32;
  // how a launch splits it, set by plan_heads
  int shift;   // log2 of the groups side by side on one token's heads
  int tokens;  // of a tile
  int blocks;
  long long tiles;
};

struct HeadArgs {
  HeadOp op[2];
  const void* positions;
  const int* axis_of;  // [pairs] or nullptr
  const void* freq;    // [pairs] fp32 or fp64
  long long axis_stride, tokens;
  int positions64, freq64, axes, pairs, start, interleaved;
  int D, type, w_type;
  float eps;
  float* part;  // workspace: [blocks][2][D] column sums
  int num_sms;
  int ring;  // where the ring of rows begins in shared memory
};

// Blocks of a backward pass at most, which is what its workspace holds.
constexpr int kHeadBlocks = 608;

cudaError_t launch_heads(const HeadArgs& a, bool backward, cudaStream_t st);
cudaError_t heads_f32(const HeadArgs& a, bool backward, cudaStream_t st);
cudaError_t heads_bf16(const HeadArgs& a, bool backward, cudaStream_t st);
cudaError_t heads_f16(const HeadArgs& a, bool backward, cudaStream_t st);

}  // namespace ibwd
