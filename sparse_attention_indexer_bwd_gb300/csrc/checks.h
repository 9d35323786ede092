// Argument checks that the C entry points of the operators share.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "indexer_train.h"
#include "train.h"

namespace ibwd {

constexpr int kMaxWidth = 1 << 30;
constexpr int64_t kMaxRows = 1LL << 27;

inline size_t size_of(int type) { return type == IBWD_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == IBWD_F32 || type == IBWD_BF16 || type == IBWD_F16; }
inline bool natural(const void* p, size_t size) { return p && (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0; }

// Shape and stride of a [rows, width] matrix.
inline int matrix_status(int64_t rows, int width, int64_t stride) {
  if (rows < 0 || width < 1 || stride < width) return IBWD_ERR_INVALID_ARG;
  if (rows > kMaxRows || width > kMaxWidth || (rows > 0 && stride > (1LL << 60) / rows)) return IBWD_ERR_UNSUPPORTED;
  return IBWD_OK;
}

struct Pointer {
  const void* p;
  size_t size;    // of an element
  bool optional;  // NULL is allowed
};

// Null and alignment checks, then (with the device) that the memory is the
// current device's; a matrix without rows may be NULL and is never dereferenced.
template <int N>
int pointers_aligned(const Pointer (&list)[N]) {
  for (const Pointer& q : list)
    if (q.p ? !natural(q.p, q.size) : !q.optional) return IBWD_ERR_INVALID_ARG;
  return IBWD_OK;
}
template <int N>
int pointers_resident(const Pointer (&list)[N], int device) {
  for (const Pointer& q : list)
    if (q.p && !device_pointer_ok(q.p, q.size, device)) return IBWD_ERR_INVALID_ARG;
  return IBWD_OK;
}

// A launch's error is this call's alone: the runtime keeps it for whoever asks
// for the last one next.
inline int done(cudaError_t e) {
  if (e == cudaSuccess) return IBWD_OK;
  cudaGetLastError();
  return IBWD_ERR_CUDA;
}

}  // namespace ibwd
