// C-ABI of the training operators: argument checks and launches.  The
// declarations, with their contracts, are in indexer_train.h.
#include <cmath>

#include "indexer_train.h"
#include "train.h"

namespace {

constexpr int kMaxWidth = 1 << 30;
constexpr int64_t kMaxRows = 1LL << 27;
constexpr int kMaxSumWidth = kMaxWidth - 64;  // with column sums: twice a padded width is an int

size_t size_of(int type) { return type == IBWD_F32 ? 4 : 2; }
bool type_ok(int type) { return type == IBWD_F32 || type == IBWD_BF16 || type == IBWD_F16; }
bool natural(const void* p, size_t size) { return p && (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0; }

// Shape and stride of a [rows, width] matrix.
int matrix_status(int64_t rows, int width, int64_t stride) {
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
    if (q.p && !ibwd::device_pointer_ok(q.p, q.size, device)) return IBWD_ERR_INVALID_ARG;
  return IBWD_OK;
}

// A launch's error is this call's alone: the runtime keeps it for whoever asks
// for the last one next.
int done(cudaError_t e) {
  if (e == cudaSuccess) return IBWD_OK;
  cudaGetLastError();
  return IBWD_ERR_CUDA;
}

bool temperature_ok(float t) { return t > 0.f && std::isfinite(t) && std::isfinite(1.f / t); }

// An output that starts where an input does must be that input, row by row.
bool in_place_ok(const void* out, int64_t out_stride, int out_type, const void* in, int64_t in_stride, int in_type) {
  return out != in || (out_stride == in_stride && out_type == in_type);
}

}  // namespace

extern "C" {

int ibwd_layer_norm_fwd(const void* x, int x_type, int64_t x_stride, const void* gamma, const void* beta, int w_type,
                        void* y, int y_type, int64_t y_stride, float* mean, float* rstd, int64_t rows, int width,
                        float eps, void* stream) {
  if (!type_ok(x_type) || !type_ok(y_type) || !type_ok(w_type)) return IBWD_ERR_INVALID_ARG;
  int rc = matrix_status(rows, width, x_stride);
  if (!rc) rc = matrix_status(rows, width, y_stride);
  if (rc) return rc;
  if (x_type != IBWD_F32 && y_type != x_type) return IBWD_ERR_UNSUPPORTED;
  if (w_type != IBWD_F32 && w_type != x_type) return IBWD_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return IBWD_ERR_INVALID_ARG;
  if (!rows) return IBWD_OK;
  const Pointer list[] = {{x, size_of(x_type), false},    {y, size_of(y_type), false}, {gamma, size_of(w_type), true},
                          {beta, size_of(w_type), true}, {mean, 4, true},             {rstd, 4, true}};
  if ((rc = pointers_aligned(list))) return rc;
  if (!in_place_ok(y, y_stride, y_type, x, x_stride, x_type)) return IBWD_ERR_INVALID_ARG;
  ibwd::NormFwdArgs a{};
  int device;
  if ((rc = ibwd::current_device(&device, &a.num_sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.N = width;
  a.x_type = x_type;
  a.y_type = y_type;
  a.w_type = w_type;
  a.eps = eps;
  return done(ibwd::launch_norm_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t ibwd_layer_norm_bwd_workspace_size(int64_t rows, int width) {
  if (matrix_status(rows, width, width) || width > kMaxSumWidth) return 0;
  return ibwd::norm_bwd_workspace(rows, width);
}

int ibwd_layer_norm_bwd(const void* dy, int dy_type, int64_t dy_stride, const void* x, int x_type, int64_t x_stride,
                        const void* gamma, int w_type, const float* mean, const float* rstd, void* dx,
                        int64_t dx_stride, float* dgamma, float* dbeta, int64_t rows, int width, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!type_ok(x_type) || !type_ok(dy_type) || !type_ok(w_type)) return IBWD_ERR_INVALID_ARG;
  int rc = matrix_status(rows, width, x_stride);
  if (!rc) rc = matrix_status(rows, width, dy_stride);
  if (!rc) rc = matrix_status(rows, width, dx_stride);
  if (rc) return rc;
  const bool sums = dgamma || dbeta;
  if (sums && width > kMaxSumWidth) return IBWD_ERR_UNSUPPORTED;
  if (x_type != IBWD_F32 && dy_type != x_type && dy_type != IBWD_F32) return IBWD_ERR_UNSUPPORTED;
  if (w_type != IBWD_F32 && w_type != x_type) return IBWD_ERR_UNSUPPORTED;
  const bool none = rows == 0;  // only the column sums are written then
  const Pointer list[] = {{dy, size_of(dy_type), none}, {x, size_of(x_type), none}, {gamma, size_of(w_type), true},
                          {mean, 4, none},              {rstd, 4, none},            {dx, size_of(x_type), none},
                          {dgamma, 4, true},            {dbeta, 4, true}};
  if ((rc = pointers_aligned(list))) return rc;
  if (!none && (!in_place_ok(dx, dx_stride, x_type, x, x_stride, x_type) ||
                !in_place_ok(dx, dx_stride, x_type, dy, dy_stride, dy_type)))
    return IBWD_ERR_INVALID_ARG;
  if (sums && !natural(workspace, 16)) return IBWD_ERR_WORKSPACE;
  ibwd::NormBwdArgs a{};
  int device;
  if ((rc = ibwd::current_device(&device, &a.num_sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  if (sums && (workspace_bytes < ibwd::norm_bwd_workspace(rows, width) || !ibwd::device_pointer_ok(workspace, 16, device)))
    return IBWD_ERR_WORKSPACE;
  a.dy = dy;
  a.x = x;
  a.gamma = gamma;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = static_cast<float*>(workspace);
  a.rows = rows;
  a.dy_stride = dy_stride;
  a.x_stride = x_stride;
  a.dx_stride = dx_stride;
  a.N = width;
  a.x_type = x_type;
  a.dy_type = dy_type;
  a.w_type = w_type;
  return done(ibwd::launch_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

int ibwd_token_logprobs_fwd(const void* logits, int type, int64_t stride, const int32_t* tokens, float temperature,
                            float* logprob, float* entropy, float* lse, int32_t* top_ids, float* top_logprobs,
                            int top_n, int64_t rows, int vocab, void* stream) {
  if (!type_ok(type) || !temperature_ok(temperature)) return IBWD_ERR_INVALID_ARG;
  int rc = matrix_status(rows, vocab, stride);
  if (rc) return rc;
  if (top_n < 0 || top_n > vocab) return IBWD_ERR_INVALID_ARG;
  if (top_n > IBWD_MAX_TOP) return IBWD_ERR_UNSUPPORTED;
  if (!rows) return IBWD_OK;
  if ((tokens == nullptr) != (logprob == nullptr)) return IBWD_ERR_INVALID_ARG;
  if ((top_n > 0) != (top_ids != nullptr) || (top_n > 0) != (top_logprobs != nullptr)) return IBWD_ERR_INVALID_ARG;
  const Pointer list[] = {{logits, size_of(type), false}, {tokens, 4, true},  {logprob, 4, true},     {entropy, 4, true},
                          {lse, 4, true},                 {top_ids, 4, true}, {top_logprobs, 4, true}};
  if ((rc = pointers_aligned(list))) return rc;
  ibwd::RowArgs a{};
  int device;
  if ((rc = ibwd::current_device(&device, &a.num_sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  a.x = logits;
  a.type = type;
  a.x_stride = stride;
  a.rows = rows;
  a.V = vocab;
  a.temperature = temperature;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.top_n = top_n;
  return done(ibwd::launch_rows(ibwd::RowOp::kLogpFwd, a, static_cast<cudaStream_t>(stream)));
}

int ibwd_token_logprobs_bwd(const void* logits, int type, int64_t stride, const int32_t* tokens, float temperature,
                            const float* lse, const float* entropy, const float* dlogprob, const float* dentropy,
                            void* dlogits, int64_t dlogits_stride, int64_t rows, int vocab, void* stream) {
  if (!type_ok(type) || !temperature_ok(temperature)) return IBWD_ERR_INVALID_ARG;
  int rc = matrix_status(rows, vocab, stride);
  if (!rc) rc = matrix_status(rows, vocab, dlogits_stride);
  if (rc) return rc;
  if (!rows) return IBWD_OK;
  if ((tokens == nullptr) != (dlogprob == nullptr) || (dentropy && !entropy)) return IBWD_ERR_INVALID_ARG;
  const Pointer list[] = {{logits, size_of(type), false}, {tokens, 4, true},   {lse, 4, false},
                          {entropy, 4, true},             {dlogprob, 4, true}, {dentropy, 4, true},
                          {dlogits, size_of(type), false}};
  if ((rc = pointers_aligned(list))) return rc;
  if (!in_place_ok(dlogits, dlogits_stride, type, logits, stride, type)) return IBWD_ERR_INVALID_ARG;
  ibwd::RowArgs a{};
  int device;
  if ((rc = ibwd::current_device(&device, &a.num_sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  a.x = logits;
  a.type = type;
  a.x_stride = stride;
  a.rows = rows;
  a.V = vocab;
  a.temperature = temperature;
  a.tokens = tokens;
  a.lse = const_cast<float*>(lse);
  a.entropy = const_cast<float*>(entropy);
  a.dlogprob = dlogprob;
  a.dentropy = dentropy;
  a.dx = dlogits;
  a.dx_stride = dlogits_stride;
  return done(ibwd::launch_rows(ibwd::RowOp::kLogpBwd, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

int distill_common(ibwd::RowOp op, const void* logits, int type, int64_t stride, const int32_t* ids,
                   const float* teacher, int K, float temperature, const float* weight, float grad_scale, float* loss,
                   float* lse, void* dlogits, int64_t dlogits_stride, int64_t rows, int vocab, void* stream) {
  const bool grad = op != ibwd::RowOp::kDistillFwd;
  if (!type_ok(type) || !temperature_ok(temperature)) return IBWD_ERR_INVALID_ARG;
  int rc = matrix_status(rows, vocab, stride);
  if (!rc && grad) rc = matrix_status(rows, vocab, dlogits_stride);
  if (rc) return rc;
  if (K < 1) return IBWD_ERR_INVALID_ARG;
  if (K > IBWD_MAX_KEPT) return IBWD_ERR_UNSUPPORTED;
  if (!std::isfinite(grad_scale)) return IBWD_ERR_INVALID_ARG;
  if (!rows) return IBWD_OK;
  const bool fwd = op == ibwd::RowOp::kDistillFwd, bwd = op == ibwd::RowOp::kDistillBwd;
  const Pointer list[] = {{logits, size_of(type), false}, {ids, 4, false},   {teacher, 4, false},
                          {weight, 4, !bwd},              {loss, 4, !fwd},   {lse, 4, !(fwd || bwd)},
                          {dlogits, size_of(type), !grad}};
  if ((rc = pointers_aligned(list))) return rc;
  if (grad && !in_place_ok(dlogits, dlogits_stride, type, logits, stride, type)) return IBWD_ERR_INVALID_ARG;
  ibwd::RowArgs a{};
  int device;
  if ((rc = ibwd::current_device(&device, &a.num_sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  a.x = logits;
  a.type = type;
  a.x_stride = stride;
  a.rows = rows;
  a.V = vocab;
  a.temperature = temperature;
  a.ids = ids;
  a.teacher = teacher;
  a.K = K;
  a.dloss = weight;
  a.grad_scale = grad_scale;
  a.loss = loss;
  a.lse = lse;
  a.dx = dlogits;
  a.dx_stride = dlogits_stride;
  return done(ibwd::launch_rows(op, a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int ibwd_distill_fwd(const void* logits, int type, int64_t stride, const int32_t* ids, const float* teacher, int K,
                     float temperature, float* loss, float* lse, int64_t rows, int vocab, void* stream) {
  return distill_common(ibwd::RowOp::kDistillFwd, logits, type, stride, ids, teacher, K, temperature, nullptr, 1.f,
                        loss, lse, nullptr, 0, rows, vocab, stream);
}

int ibwd_distill_bwd(const void* logits, int type, int64_t stride, const int32_t* ids, const float* teacher, int K,
                     float temperature, const float* lse, const float* dloss, void* dlogits, int64_t dlogits_stride,
                     int64_t rows, int vocab, void* stream) {
  return distill_common(ibwd::RowOp::kDistillBwd, logits, type, stride, ids, teacher, K, temperature, dloss, 1.f,
                        nullptr, const_cast<float*>(lse), dlogits, dlogits_stride, rows, vocab, stream);
}

int ibwd_distill_grad(const void* logits, int type, int64_t stride, const int32_t* ids, const float* teacher, int K,
                      float temperature, const float* row_weight, float grad_scale, float* loss, void* dlogits,
                      int64_t dlogits_stride, int64_t rows, int vocab, void* stream) {
  return distill_common(ibwd::RowOp::kDistillGrad, logits, type, stride, ids, teacher, K, temperature, row_weight,
                        grad_scale, loss, nullptr, dlogits, dlogits_stride, rows, vocab, stream);
}

}  // extern "C"
