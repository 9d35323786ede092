// Marshalling for Python of the norm and rotation of heads (train.py) and of
// the 8-bit cache (cache.py), as train_binding.cpp's.
#include "heads_binding.h"

#include <ATen/cuda/EmptyTensor.h>

#include <cmath>

#include "binding.h"
#include "indexer_cache.h"

namespace {

using namespace binding;

// A result of no contents yet, straight from its allocator: through the dispatcher each takes 0.2 us more.
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& of) {
  return Tensor(at::detail::empty_cuda(shape, type, of.device(), std::nullopt));
}

// A [..., heads, dim] argument whose tokens step evenly.
struct Heads {
  const Tensor* t = nullptr;
  int64_t tokens = 0, heads = 0, dim = 0, token = 0, head = 0;
  int code = 0;
  at::IntArrayRef lead() const { return t->sizes().slice(0, t->dim() - 2); }
};

Heads heads(PyObject* o, const char* name) {
  Heads h;
  const Tensor& t = tensor(o, name);
  h.t = &t;
  h.code = code_of(t.scalar_type());
  if (!t.is_cuda() || h.code < 0)
    refuse(PyExc_ValueError, name, "expected a CUDA tensor of float32, bfloat16 or float16");
  const auto size = t.sizes(), stride = t.strides();
  const int64_t dims = t.dim();
  if (dims < 2 || size[dims - 1] < 1 || size[dims - 2] < 1)
    refuse(PyExc_ValueError, name, "expected [..., heads >= 1, dim >= 1]");
  if (t.device().index() != c10::cuda::current_device())
    refuse(PyExc_ValueError, name, "expected a tensor of the current device");
  h.dim = size[dims - 1];
  h.heads = size[dims - 2];
  if (h.dim > INT_MAX || h.heads > INT_MAX) refuse(PyExc_ValueError, name, "too many heads, or too wide ones");
  h.tokens = t.numel() / (h.dim * h.heads);
  if (h.dim > 1 && stride[dims - 1] != 1) refuse(PyExc_ValueError, name, "expected unit stride along a head");
  h.head = h.heads > 1 ? stride[dims - 2] : h.dim;
  h.token = h.dim * h.heads;
  if (h.tokens == 0) return h;
  int64_t tokens = 1;
  for (int64_t d = dims - 3; d >= 0; --d) {
    if (size[d] == 1) continue;
    if (tokens == 1)
      h.token = stride[d];
    else if (stride[d] != h.token * tokens)
      refuse(PyExc_ValueError, name, "the tokens do not step evenly");
    tokens *= size[d];
  }
  return h;
}

// A second argument of the first one's tokens (and heads) and device.
Heads heads_like(PyObject* o, const char* name, const Heads& of, bool same_heads) {
  const Heads h = heads(o, name);
  if (h.lead() != of.lead() || h.dim != of.dim || (same_heads && h.heads != of.heads))
    refuse(PyExc_ValueError, name, "expected the tokens, heads and width of the other argument");
  return h;
}

// A result of the shape of `of`: contiguous, or as given.
struct HeadsOut {
  Tensor t;
  int64_t token, head;
  bool given = false;
  void written() const {
    if (given && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
};
HeadsOut heads_out(PyObject* o, const char* name, const Heads& of) {
  if (o == Py_None)
    return {fresh(of.t->sizes(), of.t->scalar_type(), *of.t), of.heads * of.dim, of.dim};
  const Heads h = heads_like(o, name, of, true);
  if (h.code != of.code) refuse(PyExc_ValueError, name, "expected the type of the input");
  return {*h.t, h.token, h.head, true};
}

int norm_of(PyObject* o, const char* name) {
  const long v = integer(o);
  if (v < IBWD_NORM_NONE || v > IBWD_NORM_LAYER) refuse(PyExc_ValueError, name, "expected 'none', 'rms' or 'layer'");
  return (int)v;
}

// The weights q_gamma, q_beta, k_gamma, k_beta at a[0..3]: float32 or the heads' type, all alike.
int head_weights(const Heads& q, PyObject* const* a, const void* (&p)[4]) {
  static const char* const names[] = {"q_gamma", "q_beta", "k_gamma", "k_beta"};
  auto type = at::kFloat;
  for (int i = 0; i < 4; ++i)
    if (a[i] != Py_None) {
      type = tensor(a[i], names[i]).scalar_type();
      break;
    }
  if (type != at::kFloat && type != q.t->scalar_type())
    refuse(PyExc_ValueError, "the weights", "expected float32 or the type of the heads");
  for (int i = 0; i < 4; ++i) p[i] = like_or_null(a[i], names[i], {}, q.dim, type, *q.t);
  return code_of(type);
}

// positions, inv_freq, axes, start, interleaved at a[0..4]
ibwd_rotation rotation(const Heads& q, PyObject* const* a) {
  ibwd_rotation r{};
  if ((a[0] == Py_None) != (a[1] == Py_None)) refuse(PyExc_ValueError, "positions", "go together with inv_freq");
  if (a[0] == Py_None) return r;
  const Tensor &p = tensor(a[0], "positions"), &f = tensor(a[1], "inv_freq");
  if (p.scalar_type() != at::kInt && p.scalar_type() != at::kLong)
    refuse(PyExc_ValueError, "positions", "expected int32 or int64");
  if (f.scalar_type() != at::kFloat && f.scalar_type() != at::kDouble)
    refuse(PyExc_ValueError, "inv_freq", "expected float32 or float64");
  if (f.dim() != 1 || f.size(0) > INT_MAX / 2) refuse(PyExc_ValueError, "inv_freq", "expected one value a pair");
  r.pairs = (int)f.size(0);
  r.freq = like(a[1], "inv_freq", {}, r.pairs, f.scalar_type(), *q.t);
  r.freq_f64 = f.scalar_type() == at::kDouble;
  r.positions_int64 = p.scalar_type() == at::kLong;
  r.axes = 1;
  std::vector<int64_t> shape = q.lead().vec();
  if (a[2] != Py_None) {
    if (p.dim() != (int64_t)shape.size() + 1 || p.size(0) < 1 || p.size(0) > INT_MAX)
      refuse(PyExc_ValueError, "positions", "expected [axes, ...] beside the tokens");
    r.axes = (int)p.size(0);
    shape.insert(shape.begin(), p.size(0));
    r.axis_of = static_cast<const int32_t*>(like(a[2], "axes", {}, r.pairs, at::kInt, *q.t));
  }
  r.positions = like(a[0], "positions", shape, -1, p.scalar_type(), *q.t);
  if (!r.pairs) r.positions = nullptr;
  r.axis_stride = q.tokens;
  const long start = integer(a[3]);
  if (start < 0 || start > INT_MAX) refuse(PyExc_ValueError, "start", "beyond the heads");
  r.start = (int)start;
  r.interleaved = a[4] == Py_True;
  return r;
}

ibwd_heads operand(const Heads& h, int norm, const void* gamma, const HeadsOut& out) {
  ibwd_heads r{};
  r.x = h.t->const_data_ptr();
  r.x_token = h.token;
  r.x_head = h.head;
  r.heads = (int)h.heads;
  r.norm = norm;
  r.gamma = gamma;
  r.y = out.t.data_ptr();
  r.y_token = out.token;
  r.y_head = out.head;
  return r;
}

// Keys of the other type than the queries, and a k_* argument without keys.
void no_keys(PyObject* o, const char* name) {
  if (o != Py_None) refuse(PyExc_ValueError, name, "there are no keys");
}

// The packed tokens' sequences and the shape of the caches: page_table, lens, cu.
struct Seqs : ibwd_sequences {
  Seqs() : ibwd_sequences{} {}
};
const Tensor& int32_of(PyObject* o, const char* name, int64_t dims, const Tensor& of) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt || t.dim() != dims || t.device() != of.device())
    refuse(PyExc_ValueError, name, "expected an int32 tensor of the cache's device and other dimensions");
  return t;
}
Seqs sequences(const Tensor& cache, PyObject* table, PyObject* lens, PyObject* cu) {
  Seqs s;
  const Tensor& t = int32_of(table, "page_table", 2, cache);
  if (t.size(1) > INT_MAX || t.size(0) > INT_MAX || (t.size(1) > 1 && t.stride(1) != 1))
    refuse(PyExc_ValueError, "page_table", "expected [sequences, pages] with unit stride");
  s.table = t.const_data_ptr<int32_t>();
  s.table_width = (int)t.size(1);
  s.table_stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
  s.batch = (int)t.size(0);
  s.lens = static_cast<const int32_t*>(like(lens, "lens", {t.size(0)}, -1, at::kInt, cache));
  s.cu = static_cast<const int32_t*>(like_or_null(cu, "cu", {t.size(0) + 1}, -1, at::kInt, cache));
  s.pages = cache.size(0);
  s.heads = (int)cache.size(1);
  s.page = (int)cache.size(2);
  s.dim = (int)cache.size(3);
  s.code = cache.scalar_type() == at::kChar ? IBWD_INT8 : IBWD_E4M3;
  return s;
}
// A cache's codes; the other one beside it where `beside` is given.
const Tensor& codes(PyObject* o, const char* name, const Tensor* beside) {
  const Tensor& t = tensor(o, name);
  if (!t.is_cuda() || (t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kChar) || t.dim() != 4 ||
      !t.is_contiguous())
    refuse(PyExc_ValueError, name, "expected a contiguous CUDA tensor [pages, heads, page, dim] of float8_e4m3fn or int8");
  if (t.device().index() != c10::cuda::current_device())
    refuse(PyExc_ValueError, name, "expected a tensor of the current device");
  for (int64_t n : t.sizes())
    if (n > INT_MAX) refuse(PyExc_ValueError, name, "too large");
  if (beside && (t.sizes() != beside->sizes() || t.scalar_type() != beside->scalar_type() || t.device() != beside->device()))
    refuse(PyExc_ValueError, name, "expected the shape, type and device of the keys' cache");
  return t;
}
ibwd_cache cache_of(const Tensor& t, PyObject* scale, const char* name) {
  return {t.data_ptr(),
          static_cast<float*>(const_cast<void*>(like(scale, name, t.sizes().slice(0, 2), -1, at::kFloat, t)))};
}
void bump(PyObject* o) {
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

}  // namespace

// (q, k, positions, inv_freq, axes, start, interleaved, q_norm, k_norm, q_gamma, q_beta, k_gamma, k_beta, eps, q_out, k_out)
PyObject* qk_norm_rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 16);
    const Heads q = heads(a[0], "q");
    Heads k;
    const bool keys = a[1] != Py_None;
    if (keys) {
      k = heads_like(a[1], "k", q, false);
      if (k.code != q.code) refuse(PyExc_ValueError, "k", "expected the type of q");
    } else {
      no_keys(a[11], "k_gamma");
      no_keys(a[12], "k_beta");
      no_keys(a[15], "k_out");
    }
    if (q.dim > IBWD_MAX_HEAD_DIM) refuse(PyExc_ValueError, "q", "the heads are too wide");
    const ibwd_rotation r = rotation(q, a + 2);
    const int qn = norm_of(a[7], "q_norm"), kn = norm_of(a[8], "k_norm");
    const void* w[4];
    const int wt = head_weights(q, a + 9, w);
    const float eps = number(a[13]);
    HeadsOut yq = heads_out(a[14], "q_out", q), yk;
    if (keys) yk = heads_out(a[15], "k_out", k);
    ibwd_heads oq = operand(q, qn, w[0], yq), ok{};
    oq.beta = w[1];
    if (keys) {
      ok = operand(k, kn, w[2], yk);
      ok.beta = w[3];
    }
    call("ibwd_qk_norm_rope_fwd", ibwd_qk_norm_rope_fwd, &oq, keys ? &ok : nullptr, &r, q.code, wt, q.tokens, (int)q.dim, eps,
         stream_of(*q.t));
    yq.written();
    if (keys) yk.written();
    return tuple_of(std::move(yq.t), std::move(yk.t));
  });
}

// (dyq, dyk, q, k, positions, inv_freq, axes, start, interleaved, q_norm, k_norm, q_gamma, k_gamma, eps, q_out, k_out,
//  weight_grads, workspace)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 18);
    const Heads q = heads(a[2], "q"), dq = heads_like(a[0], "dyq", q, true);
    Heads k, dk;
    const bool keys = a[3] != Py_None;
    if (keys) {
      k = heads_like(a[3], "k", q, false);
      if (k.code != q.code) refuse(PyExc_ValueError, "k", "expected the type of q");
      dk = heads_like(a[1], "dyk", k, true);
    } else {
      no_keys(a[1], "dyk");
      no_keys(a[12], "k_gamma");
      no_keys(a[15], "k_out");
    }
    if (q.dim > IBWD_MAX_HEAD_DIM) refuse(PyExc_ValueError, "q", "the heads are too wide");
    if (a[17] != Py_None && !tensor(a[17], "workspace").is_contiguous())
      refuse(PyExc_ValueError, "workspace", "expected a contiguous tensor");
    const ibwd_rotation r = rotation(q, a + 4);
    const int qn = norm_of(a[9], "q_norm"), kn = norm_of(a[10], "k_norm");
    PyObject* const given[4] = {a[11], Py_None, a[12], Py_None};
    const void* w[4];
    const int wt = head_weights(q, given, w);
    const float eps = number(a[13]);
    HeadsOut xq = heads_out(a[14], "q_out", q), xk;
    if (keys) xk = heads_out(a[15], "k_out", k);
    Tensor sums[4], work;
    auto backward = [&](const Heads& h, const Heads& dy, int norm, const void* gamma, const HeadsOut& out, int at) {
      ibwd_heads o = operand(h, norm, gamma, out);
      o.dy = dy.t->const_data_ptr();
      o.dy_type = dy.code;
      o.dy_token = dy.token;
      o.dy_head = dy.head;
      if (a[16] == Py_True && norm != IBWD_NORM_NONE) {
        sums[at] = fresh({h.dim}, at::kFloat, *h.t);
        if (norm == IBWD_NORM_LAYER) sums[at + 1] = fresh({h.dim}, at::kFloat, *h.t);
        o.dgamma = data<float>(sums[at]);
        o.dbeta = data<float>(sums[at + 1]);
      }
      return o;
    };
    const ibwd_heads oq = backward(q, dq, qn, w[0], xq, 0);
    ibwd_heads ok{};
    if (keys) ok = backward(k, dk, kn, w[2], xk, 2);
    void* ws = nullptr;
    size_t bytes = 0;
    if (sums[0].defined() || sums[2].defined()) {
      work = a[17] == Py_None ? fresh({(int64_t)ibwd_qk_norm_rope_bwd_workspace_size((int)q.dim)}, at::kByte, *q.t)
                              : tensor(a[17], "workspace");
      ws = work.data_ptr();
      bytes = work.nbytes();
    }
    call("ibwd_qk_norm_rope_bwd", ibwd_qk_norm_rope_bwd, &oq, keys ? &ok : nullptr, &r, q.code, wt, q.tokens, (int)q.dim, eps,
         ws, bytes, stream_of(*q.t));
    xq.written();
    if (keys) xk.written();
    return tuple_of(std::move(xq.t), std::move(xk.t), std::move(sums[0]), std::move(sums[1]), std::move(sums[2]),
                    std::move(sums[3]));
  });
}

// (k, v, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 9);
    const Tensor& kc = codes(a[2], "k_cache", nullptr);
    const Heads k = heads(a[0], "k");
    const bool values = a[1] != Py_None;
    if (values != (a[3] != Py_None) || values != (a[5] != Py_None))
      refuse(PyExc_ValueError, "v", "goes together with v_cache and v_scale");
    Heads v;
    ibwd_cache ck = cache_of(kc, a[4], "k_scale"), cv{};
    if (values) {
      v = heads_like(a[1], "v", k, true);
      if (v.code != k.code) refuse(PyExc_ValueError, "v", "expected the type of k");
      cv = cache_of(codes(a[3], "v_cache", &kc), a[5], "v_scale");
    }
    Seqs s = sequences(kc, a[6], a[7], a[8]);
    if (k.heads != s.heads || k.dim != s.dim) refuse(PyExc_ValueError, "k", "expected the cache's heads");
    s.tokens = k.tokens;
    call("ibwd_cache_write", ibwd_cache_write, k.t->const_data_ptr(), k.token, k.head,
         values ? v.t->const_data_ptr() : nullptr, v.token, v.head, k.code, &ck, values ? &cv : nullptr, &s, stream_of(kc));
    bump(a[2]);
    bump(a[4]);
    if (values) {
      bump(a[3]);
      bump(a[5]);
    }
    Py_RETURN_NONE;
  });
}

// (cache, scale, page_table, lens, length, type code, out)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    const Tensor& c = codes(a[0], "cache", nullptr);
    const ibwd_cache from = cache_of(c, a[1], "scale");
    Seqs s = sequences(c, a[2], a[3], Py_None);
    const long length = integer(a[4]);
    if (length < 0 || length > INT_MAX) refuse(PyExc_ValueError, "length", "out of range");
    const int code = (int)integer(a[5]);
    const int64_t shape[4] = {s.batch, length, s.heads, s.dim};
    Tensor out;
    const bool given = a[6] != Py_None;
    if (given) {
      like(a[6], "out", shape, -1, type_of(code), c);
      out = tensor(a[6], "out");
    } else {
      out = fresh(shape, type_of(code), c);
    }
    call("ibwd_cache_read", ibwd_cache_read, &from, &s, out.data_ptr(), code, (int)length, stream_of(c));
    if (given) bump(a[6]);
    return wrap(std::move(out));
  });
}

// (q, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu, select, scale or None, workspace, out)
PyObject* cache_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 12);
    const Tensor& kc = codes(a[1], "k_cache", nullptr);
    const ibwd_cache ck = cache_of(kc, a[3], "k_scale"), cv = cache_of(codes(a[2], "v_cache", &kc), a[4], "v_scale");
    const Heads q = heads(a[0], "q");
    Seqs s = sequences(kc, a[5], a[6], a[7]);
    if (q.dim != s.dim || s.heads < 1 || q.heads % s.heads)
      refuse(PyExc_ValueError, "q", "expected the cache's width and a multiple of its heads");
    s.tokens = q.tokens;
    const int32_t* select = nullptr;
    int kept = 0;
    if (a[8] != Py_None) {
      const Tensor& t = tensor(a[8], "select");
      if (t.dim() < 1 || t.size(t.dim() - 1) > INT_MAX) refuse(PyExc_ValueError, "select", "expected [..., kept]");
      kept = (int)t.size(t.dim() - 1);
      select = static_cast<const int32_t*>(like(a[8], "select", q.lead(), kept, at::kInt, *q.t));
      if (!kept) refuse(PyExc_ValueError, "select", "expected at least one place");
    }
    const float scale = a[9] == Py_None ? 1.f / std::sqrt((float)q.dim) : number(a[9]);
    Tensor work, out, lse;
    if (a[10] == Py_None) {
      work = fresh({(int64_t)ibwd_cache_attention_workspace_size(s.dim)}, at::kByte, kc);
    } else {
      work = tensor(a[10], "workspace");
      if (!work.is_contiguous()) refuse(PyExc_ValueError, "workspace", "expected a contiguous tensor");
    }
    const bool given = a[11] != Py_None;
    if (given) {
      like(a[11], "out", q.t->sizes(), -1, q.t->scalar_type(), *q.t);
      out = tensor(a[11], "out");
    } else {
      out = fresh(q.t->sizes(), q.t->scalar_type(), *q.t);
    }
    std::vector<int64_t> rows = q.lead().vec();
    rows.push_back(q.heads);
    lse = fresh(rows, at::kFloat, *q.t);
    call("ibwd_cache_attention", ibwd_cache_attention, q.t->const_data_ptr(), q.token, q.head, q.code,
         (int)(q.heads / s.heads), &ck, &cv, &s, select, kept, scale, out.data_ptr(), data<float>(lse), work.data_ptr(),
         work.nbytes(), stream_of(kc));
    if (given) bump(a[11]);
    return tuple_of(std::move(out), std::move(lse));
  });
}
