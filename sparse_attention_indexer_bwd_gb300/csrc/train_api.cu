// C-ABI of the training operators: argument checks and launches.  The
// declarations, with their contracts, are in indexer_train.h.
#include <cmath>

#include "checks.h"
#include "head_norm.h"

namespace {

using namespace ibwd;

constexpr int kMaxSumWidth = kMaxWidth - 64;  // with column sums: twice a padded width is an int

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

namespace {

bool any_sum(const ibwd_heads* q) { return q && q->heads > 0 && (q->dgamma || q->dbeta); }

// Steps between a result's tokens and heads: any that do not overlap, whatever their order.
bool steps_ok(int64_t token, int64_t head, int64_t tokens, int heads, int dim) {
  if (token < 0 || head < 0) return false;
  if (heads > 1 && head < dim) return false;
  if (tokens > 1 && token < dim) return false;
  if (tokens <= 1 || heads <= 1) return true;
  return token >= (heads - 1) * head + dim || head >= (tokens - 1) * token + dim;
}
bool steps_far(int64_t token, int64_t head, int64_t tokens, int heads) {
  constexpr int64_t far = 1LL << 58;
  return (tokens > 1 && token > far / tokens) || (heads > 1 && head > far / heads);
}

// Checks one operand; fills `o` and appends its pointers to `list`.
int head_op(const ibwd_heads& h, bool backward, int type, int w_type, int64_t tokens, int dim, bool none, HeadOp* o,
            Pointer* list, int* n) {
  if (h.heads < 0) return IBWD_ERR_INVALID_ARG;
  if (!h.heads) return IBWD_OK;
  if (h.heads > 1 << 16) return IBWD_ERR_UNSUPPORTED;
  if (h.norm != IBWD_NORM_NONE && h.norm != IBWD_NORM_RMS && h.norm != IBWD_NORM_LAYER) return IBWD_ERR_INVALID_ARG;
  if ((h.gamma && h.norm == IBWD_NORM_NONE) || (h.beta && h.norm != IBWD_NORM_LAYER)) return IBWD_ERR_INVALID_ARG;
  if (steps_far(h.x_token, h.x_head, tokens, h.heads) || steps_far(h.y_token, h.y_head, tokens, h.heads) ||
      (backward && steps_far(h.dy_token, h.dy_head, tokens, h.heads)))
    return IBWD_ERR_UNSUPPORTED;
  if (h.x_token < 0 || h.x_head < 0 || !steps_ok(h.y_token, h.y_head, tokens, h.heads, dim)) return IBWD_ERR_INVALID_ARG;
  const size_t size = size_of(type);
  list[(*n)++] = {h.x, size, none || (backward && h.norm == IBWD_NORM_NONE)};
  list[(*n)++] = {h.y, size, none};
  list[(*n)++] = {h.gamma, size_of(w_type), true};
  if (!backward) list[(*n)++] = {h.beta, size_of(w_type), true};
  if (h.y == h.x && h.y && (h.y_token != h.x_token || h.y_head != h.x_head)) return IBWD_ERR_INVALID_ARG;
  if (backward) {
    if (h.dy_type != type && h.dy_type != IBWD_F32) return type_ok(h.dy_type) ? IBWD_ERR_UNSUPPORTED : IBWD_ERR_INVALID_ARG;
    // (a gradient that several heads or tokens share may have steps of 0)
    if (h.dy_token < 0 || h.dy_head < 0) return IBWD_ERR_INVALID_ARG;
    if ((h.dgamma && h.norm == IBWD_NORM_NONE) || (h.dbeta && h.norm != IBWD_NORM_LAYER)) return IBWD_ERR_INVALID_ARG;
    list[(*n)++] = {h.dy, size_of(h.dy_type), none};
    list[(*n)++] = {h.dgamma, 4, true};
    list[(*n)++] = {h.dbeta, 4, true};
    if (h.y == h.dy && h.y && (h.y_token != h.dy_token || h.y_head != h.dy_head || h.dy_type != type))
      return IBWD_ERR_INVALID_ARG;
    o->dy = h.dy;
    o->dy_token = h.dy_token;
    o->dy_head = h.dy_head;
    o->dy_f32 = h.dy_type == IBWD_F32;
    o->dgamma = h.dgamma;
    o->dbeta = h.dbeta;
  } else {
    o->beta = h.beta;
  }
  o->x = h.x;
  o->y = h.y;
  o->gamma = h.gamma;
  o->x_token = h.x_token;
  o->x_head = h.x_head;
  o->y_token = h.y_token;
  o->y_head = h.y_head;
  o->heads = h.heads;
  o->norm = h.norm;
  return IBWD_OK;
}

int heads_common(bool backward, const ibwd_heads* q, const ibwd_heads* k, const ibwd_rotation* r, int type, int w_type,
                 int64_t tokens, int dim, float eps, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !type_ok(type) || !type_ok(w_type) || tokens < 0 || dim < 1) return IBWD_ERR_INVALID_ARG;
  if (tokens > kMaxRows || dim > IBWD_MAX_HEAD_DIM || (w_type != IBWD_F32 && w_type != type)) return IBWD_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return IBWD_ERR_INVALID_ARG;
  const bool none = tokens == 0;  // only the weights' sums are written then
  HeadArgs a{};
  Pointer list[17];
  int n = 0, rc = head_op(*q, backward, type, w_type, tokens, dim, none, &a.op[0], list, &n);
  if (!rc && k) rc = head_op(*k, backward, type, w_type, tokens, dim, none, &a.op[1], list, &n);
  if (rc) return rc;
  if (a.op[0].heads && a.op[1].heads && !none) {  // one operand's result is nothing of the other's
    const HeadOp &o = a.op[0], &p = a.op[1];
    if (o.y == p.y || o.y == p.x || p.y == o.x || (backward && (o.y == p.dy || p.y == o.dy))) return IBWD_ERR_INVALID_ARG;
  }
  if (backward) {
    const float* const to[4] = {a.op[0].dgamma, a.op[0].dbeta, a.op[1].dgamma, a.op[1].dbeta};
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < i; ++j)
        if (to[i] && to[i] == to[j]) return IBWD_ERR_INVALID_ARG;
  }
  if (r && r->positions) {
    if (r->pairs < 0 || r->start < 0 || r->axes < 1 || r->pairs > dim / 2 || r->start > dim - 2 * r->pairs)
      return IBWD_ERR_INVALID_ARG;
    if (r->axes > 8) return IBWD_ERR_UNSUPPORTED;
    if (r->axes > 1 && (r->axis_stride < tokens || r->axis_stride > (1LL << 40))) return IBWD_ERR_INVALID_ARG;
    if (r->pairs) {
      list[n++] = {r->positions, r->positions_int64 ? 8u : 4u, none};
      list[n++] = {r->freq, r->freq_f64 ? 8u : 4u, none};
      list[n++] = {r->axis_of, 4, true};
    }
    a.positions = r->positions;
    a.positions64 = r->positions_int64;
    a.axis_stride = r->axis_stride;
    a.axes = r->axes;
    a.axis_of = r->axis_of;
    a.freq = r->freq;
    a.freq64 = r->freq_f64;
    a.pairs = r->pairs;
    a.start = r->start;
    a.interleaved = r->interleaved != 0;
  }
  const bool sums = backward && (any_sum(q) || any_sum(k));
  if (none && !sums) return IBWD_OK;
  for (int i = 0; i < n; ++i)
    if (list[i].p ? !natural(list[i].p, list[i].size) : !list[i].optional) return IBWD_ERR_INVALID_ARG;
  if (sums && !natural(workspace, 16)) return IBWD_ERR_WORKSPACE;
  int device;
  if ((rc = current_device(&device, &a.num_sms))) return rc;
  for (int i = 0; i < n; ++i)
    if (list[i].p && !device_pointer_ok(list[i].p, list[i].size, device)) return IBWD_ERR_INVALID_ARG;
  if (sums && (workspace_bytes < ibwd_qk_norm_rope_bwd_workspace_size(dim) || !device_pointer_ok(workspace, 16, device)))
    return IBWD_ERR_WORKSPACE;
  a.tokens = tokens;
  a.D = dim;
  a.type = type;
  a.w_type = w_type;
  a.eps = eps;
  a.part = static_cast<float*>(workspace);
  return done(launch_heads(a, backward, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int ibwd_qk_norm_rope_fwd(const ibwd_heads* q, const ibwd_heads* k, const ibwd_rotation* rotation, int type, int w_type,
                          int64_t tokens, int dim, float eps, void* stream) {
  return heads_common(false, q, k, rotation, type, w_type, tokens, dim, eps, nullptr, 0, stream);
}

size_t ibwd_qk_norm_rope_bwd_workspace_size(int dim) {
  return dim < 1 || dim > IBWD_MAX_HEAD_DIM ? 0 : (size_t)kHeadBlocks * 2 * dim * 4;
}

int ibwd_qk_norm_rope_bwd(const ibwd_heads* q, const ibwd_heads* k, const ibwd_rotation* rotation, int type, int w_type,
                          int64_t tokens, int dim, float eps, void* workspace, size_t workspace_bytes, void* stream) {
  return heads_common(true, q, k, rotation, type, w_type, tokens, dim, eps, workspace, workspace_bytes, stream);
}

}  // extern "C"
