// C-ABI of the 8-bit cache and the attention over it: argument checks and
// launches. The declarations, with their contracts, are in indexer_cache.h.
#include <climits>
#include <cmath>

#include "cache.h"
#include "checks.h"
#include "indexer_cache.h"

namespace {

using namespace ibwd;

// The shape of the sequences and of the caches; fills `s`.
int seqs_status(const ibwd_sequences* q, CacheSeqs* s) {
  if (!q || q->batch < 0 || q->table_width < 1 || q->pages < 1 || q->heads < 1 || q->dim < 1 || q->page < 1 || q->tokens < 0 ||
      (q->batch > 1 && q->table_stride < q->table_width) || (q->code != IBWD_E4M3 && q->code != IBWD_INT8))
    return IBWD_ERR_INVALID_ARG;
  if (q->page < 16 || q->page > 256 || (q->page & (q->page - 1)) || q->dim % 16 || q->dim > IBWD_MAX_HEAD_DIM ||
      q->heads > 65535 || q->batch > 1 << 20 || q->tokens > kMaxRows || q->pages > INT_MAX ||
      q->table_width > INT_MAX / q->page || q->table_stride > 1LL << 40)
    return IBWD_ERR_UNSUPPORTED;
  s->table = q->table;
  s->lens = q->lens;
  s->cu = q->cu;
  s->stride = q->table_stride;
  s->pages = q->pages;
  s->tokens = q->tokens;
  s->batch = q->batch;
  s->width = q->table_width;
  s->page_log = 0;
  while ((1 << s->page_log) < q->page) ++s->page_log;
  return IBWD_OK;
}

// A [tokens, heads, dim] argument's steps.
int heads_status(int64_t token, int64_t head, int64_t tokens, int64_t heads) {
  if (token < 0 || head < 0) return IBWD_ERR_INVALID_ARG;
  constexpr int64_t far = 1LL << 58;
  return (tokens > 1 && token > far / tokens) || (heads > 1 && head > far / heads) ? IBWD_ERR_UNSUPPORTED : IBWD_OK;
}

Pointer codes_of(const ibwd_cache* c) { return {c ? c->codes : nullptr, 16, false}; }
Pointer scale_of(const ibwd_cache* c) { return {c ? c->scale : nullptr, 4, false}; }

}  // namespace

extern "C" {

int ibwd_cache_write(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head, int type,
                     const ibwd_cache* k_cache, const ibwd_cache* v_cache, const ibwd_sequences* seqs, void* stream) {
  CacheWriteArgs a{};
  int rc = seqs_status(seqs, &a.seqs);
  if (rc) return rc;
  if (!type_ok(type) || (v == nullptr) != (v_cache == nullptr)) return IBWD_ERR_INVALID_ARG;
  if ((rc = heads_status(k_token, k_head, seqs->tokens, seqs->heads))) return rc;
  if (v && (rc = heads_status(v_token, v_head, seqs->tokens, seqs->heads))) return rc;
  // without offsets the packed tokens are one a sequence
  if (!seqs->cu && seqs->tokens != seqs->batch) return IBWD_ERR_INVALID_ARG;
  if (!seqs->tokens || !seqs->batch) return IBWD_OK;
  const size_t size = size_of(type);
  const Pointer none{nullptr, 4, true};
  const Pointer list[] = {{k, size, false},      {v, size, true},      codes_of(k_cache),       scale_of(k_cache),
                          v ? codes_of(v_cache) : none, v ? scale_of(v_cache) : none, {seqs->table, 4, false},
                          {seqs->lens, 4, false}, {seqs->cu, 4, true}};
  if ((rc = pointers_aligned(list))) return rc;
  if (v && (v_cache->codes == k_cache->codes || v_cache->scale == k_cache->scale)) return IBWD_ERR_INVALID_ARG;
  int device, sms;
  if ((rc = current_device(&device, &sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  a.x[0] = k;
  a.x[1] = v;
  a.token[0] = k_token;
  a.token[1] = v_token;
  a.head[0] = k_head;
  a.head[1] = v_head;
  a.codes[0] = k_cache->codes;
  a.scale[0] = k_cache->scale;
  a.codes[1] = v ? v_cache->codes : nullptr;
  a.scale[1] = v ? v_cache->scale : nullptr;
  a.type = type;
  a.code = seqs->code;
  a.heads = seqs->heads;
  a.dim = seqs->dim;
  return done(launch_cache_write(a, static_cast<cudaStream_t>(stream)));
}

int ibwd_cache_read(const ibwd_cache* cache, const ibwd_sequences* seqs, void* out, int type, int length, void* stream) {
  CacheReadArgs a{};
  int rc = seqs_status(seqs, &a.seqs);
  if (rc) return rc;
  if (!type_ok(type) || length < 0) return IBWD_ERR_INVALID_ARG;
  if ((long long)seqs->batch * (((long long)length + seqs->page - 1) / seqs->page) > INT_MAX ||
      length > INT_MAX - seqs->page)
    return IBWD_ERR_UNSUPPORTED;
  if (!seqs->batch || !length) return IBWD_OK;
  const Pointer list[] = {codes_of(cache), scale_of(cache), {out, 16, false}, {seqs->table, 4, false}, {seqs->lens, 4, false}};
  if ((rc = pointers_aligned(list))) return rc;
  int device, sms;
  if ((rc = current_device(&device, &sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  a.codes = cache->codes;
  a.scale = cache->scale;
  a.out = out;
  a.type = type;
  a.code = seqs->code;
  a.heads = seqs->heads;
  a.dim = seqs->dim;
  a.length = length;
  return done(launch_cache_read(a, static_cast<cudaStream_t>(stream)));
}

size_t ibwd_cache_attention_workspace_size(int dim) {
  return dim == 64 || dim == 128 || dim == 256 ? cache_attention_workspace(dim) : 0;
}

int ibwd_cache_attention(const void* q, int64_t q_token, int64_t q_head, int type, int group, const ibwd_cache* k_cache,
                         const ibwd_cache* v_cache, const ibwd_sequences* seqs, const int32_t* select, int kept, float scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  CacheAttnArgs a{};
  int rc = seqs_status(seqs, &a.seqs);
  if (rc) return rc;
  if (!type_ok(type) || group < 1 || !std::isfinite(scale * 1.44269504088896341f) || (select && kept < 1)) return IBWD_ERR_INVALID_ARG;
  if (type == IBWD_F32 || !ibwd_cache_attention_workspace_size(seqs->dim) || group > 65535 || (select && kept > 1 << 30) ||
      (long long)seqs->heads * group > INT_MAX)
    return IBWD_ERR_UNSUPPORTED;
  // Rows of a KV head, and tiles of the whole call at most: row tiles are of 16 rows at least, tiles of 64 positions, and an
  // item costs two tiles more. A block counts its share of them, a 304th or less, in an int.
  const double rows = (double)seqs->tokens * group, places = select ? kept : (double)seqs->table_width * seqs->page;
  const double ragged = (double)(select || seqs->batch > seqs->tokens ? seqs->tokens : seqs->batch);
  if (rows > 1 << 30 || (rows / 16 + ragged) * seqs->heads * (places / 64 + 3) > 300. * INT_MAX) return IBWD_ERR_UNSUPPORTED;
  if ((rc = heads_status(q_token, q_head, seqs->tokens, (int64_t)seqs->heads * group))) return rc;
  if (!seqs->cu && seqs->tokens != seqs->batch) return IBWD_ERR_INVALID_ARG;
  if (!seqs->tokens || !seqs->batch) return IBWD_OK;
  const Pointer list[] = {{q, 2, false},          codes_of(k_cache),      scale_of(k_cache),   codes_of(v_cache),
                          scale_of(v_cache),      {seqs->table, 4, false}, {seqs->lens, 4, false}, {seqs->cu, 4, true},
                          {select, 4, true},      {out, 16, false},       {lse, 4, true}};
  if ((rc = pointers_aligned(list))) return rc;
  if (out == q) return IBWD_ERR_INVALID_ARG;
  if (!natural(workspace, 16) || workspace_bytes < ibwd_cache_attention_workspace_size(seqs->dim)) return IBWD_ERR_WORKSPACE;
  int device;
  if ((rc = current_device(&device, &a.num_sms))) return rc;
  if ((rc = pointers_resident(list, device))) return rc;
  if (!device_pointer_ok(workspace, 16, device)) return IBWD_ERR_WORKSPACE;
  a.q = q;
  a.q_token = q_token;
  a.q_head = q_head;
  a.k = k_cache->codes;
  a.k_scale = k_cache->scale;
  a.v = v_cache->codes;
  a.v_scale = v_cache->scale;
  a.select = select;
  a.kept = kept;
  a.out = out;
  a.lse = lse;
  a.type = type;
  a.code = seqs->code;
  a.heads = seqs->heads;
  a.group = group;
  a.dim = seqs->dim;
  a.scale_log2 = scale * 1.44269504088896341f;
  a.work = workspace;
  return done(launch_cache_attention(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace ibwd {

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st) {
  if (a.dim == 64) return cache_attention_64(a, st);
  if (a.dim == 128) return cache_attention_128(a, st);
  return cache_attention_256(a, st);
}

}  // namespace ibwd
