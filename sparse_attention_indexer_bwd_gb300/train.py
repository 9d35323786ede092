"""Training operators around the indexer: layer norm, token log probabilities
and distillation from a teacher's top logits, each with its gradient
(declared in include/indexer_train.h; the functions drop the C names' ibwd_).

A matrix argument is any [..., width] CUDA tensor whose last dimension has
unit stride and whose leading dimensions step evenly (a slice of columns of a
contiguous tensor is taken as it is; nothing is copied).  Per-row arguments
and results have the leading dimensions as their shape.  Every call is
asynchronous on the current stream or on `stream=`; there the results belong
to that stream, and the arguments are recorded on it.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, load

_F32, _I32 = torch.float32, torch.int32
_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

MAX_TOP = 128
MAX_KEPT = 1024

EXPORTS = (
    "ibwd_layer_norm_fwd",
    "ibwd_layer_norm_bwd_workspace_size",
    "ibwd_layer_norm_bwd",
    "ibwd_token_logprobs_fwd",
    "ibwd_token_logprobs_bwd",
    "ibwd_distill_fwd",
    "ibwd_distill_bwd",
    "ibwd_distill_grad",
)


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the functions above."""
    p, i, f, sz, n = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
    lib.ibwd_layer_norm_fwd.argtypes = [p, i, n, p, p, i, p, i, n, p, p, n, i, f, p]
    lib.ibwd_layer_norm_bwd_workspace_size.argtypes = [n, i]
    lib.ibwd_layer_norm_bwd.argtypes = [p, i, n, p, i, n, p, i, p, p, p, n, p, p, n, i, p, sz, p]
    lib.ibwd_token_logprobs_fwd.argtypes = [p, i, n, p, f, p, p, p, p, p, i, n, i, p]
    lib.ibwd_token_logprobs_bwd.argtypes = [p, i, n, p, f, p, p, p, p, p, n, n, i, p]
    lib.ibwd_distill_fwd.argtypes = [p, i, n, p, p, i, f, p, p, n, i, p]
    lib.ibwd_distill_bwd.argtypes = [p, i, n, p, p, i, f, p, p, p, n, n, i, p]
    lib.ibwd_distill_grad.argtypes = [p, i, n, p, p, i, f, p, f, p, p, n, n, i, p]
    for name in EXPORTS:
        getattr(lib, name).restype = i
    lib.ibwd_layer_norm_bwd_workspace_size.restype = sz


# ------------------------------------------------------------- arguments ---

def _rows(t, name):
    """(rows, width, row stride) of a [..., width] matrix argument."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype not in _CODE:
        raise ValueError(f"{name}: expected a CUDA tensor of float32, bfloat16 or float16, got {t.dtype} on {t.device}")
    shape = t.shape
    if len(shape) < 2 or shape[-1] < 1:
        raise ValueError(f"{name}: expected [..., width >= 1], got {tuple(shape)}")
    width = shape[-1]
    if t.is_contiguous():
        return t.numel() // width, width, width
    stride = t.stride()
    if len(shape) == 2 and stride[1] == 1 and stride[0] >= width:
        return shape[0], width, stride[0]
    rows, step = 1, width
    for d in range(len(shape) - 2, -1, -1):
        if shape[d] == 1:
            continue
        if rows == 1:
            step = stride[d]
        elif stride[d] != step * rows:
            raise ValueError(f"{name}: rows of strides {stride} do not step evenly")
        rows *= shape[d]
    if rows and ((width > 1 and stride[-1] != 1) or step < width):
        raise ValueError(f"{name}: expected unit stride along rows that do not overlap, got strides {stride}")
    return rows, width, step


def _like(t, name, shape, dtype, device):
    """A contiguous CUDA argument of the given shape and type."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _weights(x, width, gamma, beta):
    """Type code of gamma and beta (float32 or the type of x, both alike) and their addresses."""
    dtype = _F32
    for w in (gamma, beta):
        if w is not None:
            if not isinstance(w, torch.Tensor):
                raise TypeError("gamma and beta must be torch.Tensors")
            dtype = w.dtype
            break
    if dtype != _F32 and dtype != x.dtype:
        raise ValueError(f"gamma and beta: expected float32 or {x.dtype}, got {dtype}")
    shape, device = (width,), x.device
    return (_CODE[dtype], None if gamma is None else _like(gamma, "gamma", shape, dtype, device),
            None if beta is None else _like(beta, "beta", shape, dtype, device))


def _matrix_out(out, like, dtype, name):
    """An output with the shape of `like` and its row stride: given, or allocated with the strides of `like`."""
    if out is None:
        if like.is_contiguous():
            out = torch.empty_like(like) if dtype == like.dtype else torch.empty_like(like, dtype=dtype)
        else:
            out = torch.empty_strided(like.shape, like.stride(), dtype=dtype, device=like.device)
        return out, None
    if isinstance(out, torch.Tensor) and (out.shape != like.shape or out.dtype != dtype or out.device != like.device):
        raise ValueError(f"{name}: expected {dtype} {tuple(like.shape)} on {like.device}, "
                         f"got {out.dtype} {tuple(out.shape)} on {out.device}")
    return out, _rows(out, name)[2]


def _on(stream, call, *args, **kwargs):
    """call(...) with `stream` as the current one, its arguments recorded on it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    with torch.cuda.stream(stream):
        result = call(*args, **kwargs)
    for t in (*args, *kwargs.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return result


_current_stream = torch._C._cuda_getCurrentRawStream  # the handle alone: building a Stream object takes 3 us


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------ layer norm ---

def layer_norm_fwd(x, gamma=None, beta=None, eps: float = 1e-5, out_dtype=None, out=None, stats: bool = True,
                   stream=None):
    """y = (x - mean) * rstd * gamma + beta over the last dimension.

    gamma and beta are float32 or of x's type; out_dtype (default: x's type)
    may be any type for a float32 x.  `out` may supply y, x itself among it.
    Returns (y, mean, rstd), the statistics float32 or None without `stats`."""
    if stream is not None:
        return _on(stream, layer_norm_fwd, x, gamma, beta, eps, out_dtype, out, stats)
    rows, width, xs = _rows(x, "x")
    wt, pg, pb = _weights(x, width, gamma, beta)
    dtype = out_dtype or (x.dtype if out is None else out.dtype)
    if dtype not in _CODE:
        raise ValueError(f"out_dtype: expected float32, bfloat16 or float16, got {dtype}")
    y, ys = _matrix_out(out, x, dtype, "out")
    mean = torch.empty(x.shape[:-1], dtype=_F32, device=x.device) if stats else None
    rstd = torch.empty_like(mean) if stats else None
    rc = load().ibwd_layer_norm_fwd(x.data_ptr(), _CODE[x.dtype], xs, pg, pb, wt, y.data_ptr(),
                                    _CODE[dtype], xs if ys is None else ys, _p(mean), _p(rstd), rows, width, eps,
                                    _current_stream(x.device.index))
    if rc:
        _check(rc, "ibwd_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd_workspace_size(rows: int, width: int) -> int:
    return int(load().ibwd_layer_norm_bwd_workspace_size(rows, width))


def layer_norm_bwd(dy, x, mean, rstd, gamma=None, out=None, weight_grads: bool = True, workspace=None, stream=None):
    """Backward pass of layer_norm_fwd: (dx, dgamma, dbeta), dx in x's type,
    dgamma and dbeta float32 (None without `weight_grads`).

    dy has x's type or float32 (any type for a float32 x).  `out` may supply
    dx: x, or dy where the types agree, among it."""
    if stream is not None:
        return _on(stream, layer_norm_bwd, dy, x, mean, rstd, gamma, out, weight_grads, workspace)
    rows, width, xs = _rows(x, "x")
    dyr, dyw, dys = _rows(dy, "dy")
    if dy.shape != x.shape or dy.device != x.device:
        raise ValueError(f"dy: expected {tuple(x.shape)} on {x.device}, got {tuple(dy.shape)} on {dy.device}")
    wt, pg, _ = _weights(x, width, gamma, None)
    lead = x.shape[:-1]
    pm = _like(mean, "mean", lead, _F32, x.device)
    pr = _like(rstd, "rstd", lead, _F32, x.device)
    lib = load()
    dx, dxs = _matrix_out(out, x, x.dtype, "out")
    dgamma = dbeta = None
    if weight_grads:
        dgamma = torch.empty(width, dtype=_F32, device=x.device)
        dbeta = torch.empty_like(dgamma)
        if workspace is None:
            workspace = torch.empty(lib.ibwd_layer_norm_bwd_workspace_size(rows, width), dtype=torch.uint8,
                                    device=x.device)
    rc = lib.ibwd_layer_norm_bwd(dy.data_ptr(), _CODE[dy.dtype], dys, x.data_ptr(), _CODE[x.dtype], xs, pg,
                                 wt, pm, pr, dx.data_ptr(), xs if dxs is None else dxs, _p(dgamma), _p(dbeta),
                                 rows, width, _p(workspace),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                 _current_stream(x.device.index))
    if rc:
        _check(rc, "ibwd_layer_norm_bwd")
    return dx, dgamma, dbeta


# ------------------------------------------------- token log probabilities ---

def token_logprobs_fwd(logits, tokens=None, top_n: int = 0, temperature: float = 1.0, stream=None):
    """Log probabilities of `tokens` (int32, one a row; padding outside the
    vocabulary gives 0), the rows' entropies, their log-sum-exp, and the ids
    (int32) and log probabilities of the top_n largest logits, best first.

    Returns (logprob, entropy, lse, top_ids, top_logprobs); logprob is None
    without tokens, the last two without top_n."""
    if stream is not None:
        return _on(stream, token_logprobs_fwd, logits, tokens, top_n, temperature)
    rows, vocab, step = _rows(logits, "logits")
    lead, dev = logits.shape[:-1], logits.device
    pt = None if tokens is None else _like(tokens, "tokens", lead, _I32, dev)
    entropy = torch.empty(lead, dtype=_F32, device=dev)
    lse = torch.empty_like(entropy)
    logprob = None if tokens is None else torch.empty_like(entropy)
    top_ids = top_logprobs = None
    if top_n:
        top_logprobs = torch.empty((*lead, max(0, top_n)), dtype=_F32, device=dev)
        top_ids = torch.empty_like(top_logprobs, dtype=_I32)
    rc = load().ibwd_token_logprobs_fwd(logits.data_ptr(), _CODE[logits.dtype], step, pt, temperature,
                                        _p(logprob), entropy.data_ptr(), lse.data_ptr(), _p(top_ids),
                                        _p(top_logprobs), top_n, rows, vocab, _current_stream(logits.device.index))
    if rc:
        _check(rc, "ibwd_token_logprobs_fwd")
    return logprob, entropy, lse, top_ids, top_logprobs


def token_logprobs_bwd(logits, tokens, lse, entropy=None, dlogprob=None, dentropy=None, temperature: float = 1.0,
                       out=None, stream=None):
    """Gradient of the log probabilities (dlogprob) and the entropies
    (dentropy, which needs entropy) with respect to the logits; `out` may
    supply it, the logits themselves among it."""
    if stream is not None:
        return _on(stream, token_logprobs_bwd, logits, tokens, lse, entropy, dlogprob, dentropy, temperature, out)
    rows, vocab, step = _rows(logits, "logits")
    lead, dev = logits.shape[:-1], logits.device
    if dlogprob is None:
        tokens = None  # no gradient comes through them
    pt = None if tokens is None else _like(tokens, "tokens", lead, _I32, dev)
    pl = _like(lse, "lse", lead, _F32, dev)
    pe = None if entropy is None else _like(entropy, "entropy", lead, _F32, dev)
    pd = None if dlogprob is None else _like(dlogprob, "dlogprob", lead, _F32, dev)
    ph = None if dentropy is None else _like(dentropy, "dentropy", lead, _F32, dev)
    dx, dxs = _matrix_out(out, logits, logits.dtype, "out")
    rc = load().ibwd_token_logprobs_bwd(logits.data_ptr(), _CODE[logits.dtype], step, pt, temperature, pl, pe, pd,
                                        ph, dx.data_ptr(), step if dxs is None else dxs, rows, vocab,
                                        _current_stream(logits.device.index))
    if rc:
        _check(rc, "ibwd_token_logprobs_bwd")
    return dx


# ----------------------------------------------------------- distillation ---

def _kept(logits, ids, teacher):
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dim() != logits.dim():
        raise ValueError(f"ids: expected [..., K] beside logits {tuple(logits.shape)}, got {tuple(ids.shape)}")
    shape = (*logits.shape[:-1], ids.shape[-1])
    return (_like(ids, "ids", shape, _I32, logits.device), _like(teacher, "teacher", shape, _F32, logits.device),
            shape[-1])


def distill_fwd(logits, ids, teacher, temperature: float = 1.0, stream=None):
    """Distillation loss of each row against a teacher's kept tokens: ids
    (int32 [..., K], padding outside the vocabulary) with their logits or log
    probabilities `teacher` (float32).  With p the softmax of teacher / T over
    the kept slots and q that of logits / T over the vocabulary,
    loss = T^2 sum p (log p - log q).  Returns (loss, lse)."""
    if stream is not None:
        return _on(stream, distill_fwd, logits, ids, teacher, temperature)
    rows, vocab, step = _rows(logits, "logits")
    pi, pt, k = _kept(logits, ids, teacher)
    loss = torch.empty(logits.shape[:-1], dtype=_F32, device=logits.device)
    lse = torch.empty_like(loss)
    rc = load().ibwd_distill_fwd(logits.data_ptr(), _CODE[logits.dtype], step, pi, pt, k, temperature,
                                 loss.data_ptr(), lse.data_ptr(), rows, vocab, _current_stream(logits.device.index))
    if rc:
        _check(rc, "ibwd_distill_fwd")
    return loss, lse


def distill_bwd(logits, ids, teacher, lse, dloss, temperature: float = 1.0, out=None, stream=None):
    """Gradient of distill_fwd's losses with respect to the logits, given the
    losses' own gradient dloss; `out` may supply it, the logits among it."""
    if stream is not None:
        return _on(stream, distill_bwd, logits, ids, teacher, lse, dloss, temperature, out)
    rows, vocab, step = _rows(logits, "logits")
    pi, pt, k = _kept(logits, ids, teacher)
    lead = logits.shape[:-1]
    pl = _like(lse, "lse", lead, _F32, logits.device)
    pd = _like(dloss, "dloss", lead, _F32, logits.device)
    dx, dxs = _matrix_out(out, logits, logits.dtype, "out")
    rc = load().ibwd_distill_bwd(logits.data_ptr(), _CODE[logits.dtype], step, pi, pt, k, temperature, pl, pd,
                                 dx.data_ptr(), step if dxs is None else dxs, rows, vocab, _current_stream(logits.device.index))
    if rc:
        _check(rc, "ibwd_distill_bwd")
    return dx


def distill_grad(logits, ids, teacher, row_weight=None, grad_scale: float = 1.0, temperature: float = 1.0, out=None,
                 stream=None):
    """Loss and gradient in one call: (loss, dlogits) with dlogits the
    gradient of grad_scale * sum row_weight * loss (row_weight float32, one a
    row; None for 1).  `out` may supply dlogits, the logits among it."""
    if stream is not None:
        return _on(stream, distill_grad, logits, ids, teacher, row_weight, grad_scale, temperature, out)
    rows, vocab, step = _rows(logits, "logits")
    pi, pt, k = _kept(logits, ids, teacher)
    lead = logits.shape[:-1]
    pw = None if row_weight is None else _like(row_weight, "row_weight", lead, _F32, logits.device)
    loss = torch.empty(lead, dtype=_F32, device=logits.device)
    dx, dxs = _matrix_out(out, logits, logits.dtype, "out")
    rc = load().ibwd_distill_grad(logits.data_ptr(), _CODE[logits.dtype], step, pi, pt, k, temperature, pw,
                                  grad_scale, loss.data_ptr(), dx.data_ptr(), step if dxs is None else dxs, rows,
                                  vocab, _current_stream(logits.device.index))
    if rc:
        _check(rc, "ibwd_distill_grad")
    return loss, dx
