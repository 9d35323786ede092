// Launchers of the training operators (layer norm, token log probabilities,
// distillation), shared by train_api.cu and their kernels' files.  Each
// returns a cudaError_t from its launches.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ibwd {

// The current device: IBWD_OK with its number and SM count, or the status that refuses it.
int current_device(int* device, int* num_sms);
// Whether memory of `type` that lies on device `of` may be given to a kernel
// of `device`: its own or managed memory; of any device where that is -1.
inline bool memory_fits(cudaMemoryType type, int of, int device) {
  return type == cudaMemoryTypeManaged || (type == cudaMemoryTypeDevice && (device < 0 || of == device));
}
// Non-null, aligned to `align` bytes and memory that fits.
bool device_pointer_ok(const void* p, size_t align, int device);

// Lets launches of a kernel have up to `bytes` of dynamic shared memory, once a
// device: the most that any of its launches has, since the limit is the
// process's and a smaller one would refuse another thread's launch.  `done`
// [64]: what each device's limit was raised to.
inline cudaError_t raise_smem(const void* kern, size_t bytes, std::atomic<size_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_acquire) >= bytes)) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done[dev].store(bytes, std::memory_order_release);
  return e;
}

struct NormFwdArgs {
  const void* x;
  const void* gamma;  // [N] or nullptr
  const void* beta;
  void* y;
  float* mean;  // [rows] or nullptr
  float* rstd;
  long long rows, x_stride, y_stride;
  int N, x_type, y_type, w_type;
  float eps;
  int num_sms;
};
cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t st);

struct NormBwdArgs {
  const void* dy;
  const void* x;
  const void* gamma;  // [N] or nullptr
  const float* mean;
  const float* rstd;
  void* dx;
  float* dgamma;  // [N] or nullptr
  float* dbeta;
  float* part;  // workspace: [groups][2][N rounded up to 4] column sums
  long long rows, dy_stride, x_stride, dx_stride;
  int N, x_type, dy_type, w_type;
  int num_sms;
};
cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t st);
size_t norm_bwd_workspace(long long rows, int N);
// The same by the type of x.
cudaError_t norm_fwd_f32(const NormFwdArgs& a, cudaStream_t st);
cudaError_t norm_fwd_bf16(const NormFwdArgs& a, cudaStream_t st);
cudaError_t norm_fwd_f16(const NormFwdArgs& a, cudaStream_t st);
cudaError_t norm_bwd_f32(const NormBwdArgs& a, cudaStream_t st);
cudaError_t norm_bwd_bf16(const NormBwdArgs& a, cudaStream_t st);
cudaError_t norm_bwd_f16(const NormBwdArgs& a, cudaStream_t st);

// Which function of a row of logits a launch computes.
enum class RowOp { kLogpFwd, kLogpBwd, kDistillFwd, kDistillBwd, kDistillGrad };

struct RowArgs {
  const void* x;  // logits [rows, V]
  void* dx;       // their gradient, may be x
  long long rows, x_stride, dx_stride;
  int V, type;
  float temperature;
  // log probabilities
  const int32_t* tokens;
  const float* dlogprob;
  const float* dentropy;
  float* logprob;
  float* entropy;  // written forward, read backward
  int32_t* top_ids;
  float* top_logprobs;
  int top_n;
  // distillation
  const int32_t* ids;
  const float* teacher;
  int K;
  const float* dloss;  // row weight of the gradient, or nullptr for 1
  float grad_scale;
  float* loss;
  float* lse;  // written forward, read backward
  int num_sms;
  int ahead;  // set by the launch: rows between a block's row and the next one in its place
};
cudaError_t launch_rows(RowOp op, const RowArgs& a, cudaStream_t st);
// kDistillGrad with its rows resident in shared memory, where they fit.
bool distill_resident(const RowArgs& a);
cudaError_t launch_distill_resident(const RowArgs& a, cudaStream_t st);

}  // namespace ibwd
