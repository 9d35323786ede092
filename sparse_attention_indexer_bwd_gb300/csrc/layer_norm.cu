// Layer norm: the workspace, and the choice of the type's kernels (each type of
// x is a translation unit of its own, layer_norm_*.cu).
#include "layer_norm.cuh"

namespace ibwd {

// Column sums of every group that any launch for this shape makes, on a
// device of up to kMaxSms.
size_t norm_bwd_workspace(long long rows, int N) {
  long long groups = kMaxWideGroups;
  if (N <= kMaxLateWidth) {
    // blocks of several teams, or of a team of at least N / 16 threads (with 8
    // elements each a block has more threads by more than an SM has)
    const int per_sm = N <= 32 * kElems ? bwd_per_sm(kFewElems, false) / kThreads
                                        : std::max(1, bwd_per_sm(kElems, N > kThreads * kElems) * kElems / N);
    groups = std::min<long long>(rows + 8, (long long)kMaxSms * per_sm);
    groups = std::max<long long>(groups, std::min<long long>(kMaxWideGroups, (rows + 31) / 32));
  }
  return (size_t)std::max<long long>(1, groups) * 2 * part_pitch(N) * sizeof(float);
}

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t st) {
  return a.x_type == 0 ? norm_fwd_f32(a, st) : a.x_type == 1 ? norm_fwd_bf16(a, st) : norm_fwd_f16(a, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
  return a.x_type == 0 ? norm_bwd_f32(a, st) : a.x_type == 1 ? norm_bwd_bf16(a, st) : norm_bwd_f16(a, st);
}

}  // namespace ibwd
