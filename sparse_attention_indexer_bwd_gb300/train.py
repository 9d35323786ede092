"""Training operators around the indexer: layer norm, the norm and rotation of
queries and keys, token log probabilities and distillation from a teacher's
top logits, each with its gradient (declared in include/indexer_train.h; the functions drop the C names' ibwd_).

A matrix argument is any [..., width] tensor of the current CUDA device whose
last dimension has unit stride and whose leading dimensions step evenly (a
slice of columns of a contiguous tensor is taken as it is; nothing is copied).
Per-row arguments and results have the leading dimensions as their shape.
Results of a matrix's shape are contiguous, but for rows that are no whole
16-byte blocks or do not all begin on one: those keep the input's pitch, less
whole lines of 128 bytes, so that both are read and written by vectors.

Every call is asynchronous on the current stream or on `stream=`; there the
results belong to that stream, and the arguments are recorded on it.  Autograd
does not track the calls: their gradients are the functions named after them,
and a tensor written as `out` gets a new version.

The arguments are checked and passed on by _train.so (csrc/train_binding.cpp),
a native module, because a small call takes less time on the GPU than its
marshalling did in Python: TypeError and ValueError for what is no fitting
tensor, IndexerBwdError for what the library refuses.
"""
from __future__ import annotations

import ctypes

import torch

from . import IndexerBwdError, load

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
    "ibwd_qk_norm_rope_fwd",
    "ibwd_qk_norm_rope_bwd_workspace_size",
    "ibwd_qk_norm_rope_bwd",
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
    lib.ibwd_qk_norm_rope_fwd.argtypes = [p, p, p, i, i, n, i, f, p]
    lib.ibwd_qk_norm_rope_bwd_workspace_size.argtypes = [i]
    lib.ibwd_qk_norm_rope_bwd.argtypes = [p, p, p, i, i, n, i, f, p, sz, p]
    for name in EXPORTS:
        getattr(lib, name).restype = sz if name.endswith("workspace_size") else i


_n = None  # the native module


def _native():
    global _n
    if _n is None:
        load()  # an ImportError that says how to build, where nothing is
        from . import _train
        _train.set_error(IndexerBwdError)
        _n = _train
    return _n


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


# ------------------------------------------------------------ layer norm ---

def layer_norm_fwd(x, gamma=None, beta=None, eps: float = 1e-5, out_dtype=None, out=None, stats: bool = True,
                   stream=None):
    """y = (x - mean) * rstd * gamma + beta over the last dimension.

    gamma and beta are float32 or of x's type; out_dtype (default: x's type)
    may be any type for a float32 x.  `out` may supply y, x itself among it.
    Returns (y, mean, rstd), the statistics float32 or None without `stats`."""
    if stream is not None:
        return _on(stream, layer_norm_fwd, x, gamma, beta, eps, out_dtype, out, stats)
    code = -1
    if out_dtype is not None:
        code = _CODE.get(out_dtype, -1)
        if code < 0:
            raise ValueError(f"out_dtype: expected float32, bfloat16 or float16, got {out_dtype}")
    return (_n or _native()).layer_norm_fwd(x, gamma, beta, eps, code, out, bool(stats))


def layer_norm_bwd_workspace_size(rows: int, width: int) -> int:
    if width >= 1 << 31:  # (beyond the C type, and unsupported)
        return 0
    return int(load().ibwd_layer_norm_bwd_workspace_size(rows, width))


def layer_norm_bwd(dy, x, mean, rstd, gamma=None, out=None, weight_grads: bool = True, workspace=None, stream=None):
    """Backward pass of layer_norm_fwd: (dx, dgamma, dbeta), dx in x's type,
    dgamma and dbeta float32 (None without `weight_grads`).

    dy has x's type or float32 (any type for a float32 x).  `out` may supply
    dx: x, or dy where the types agree, among it.  `workspace`: a contiguous
    tensor of layer_norm_bwd_workspace_size bytes (allocated when not given)."""
    if stream is not None:
        return _on(stream, layer_norm_bwd, dy, x, mean, rstd, gamma, out, weight_grads, workspace)
    return (_n or _native()).layer_norm_bwd(dy, x, mean, rstd, gamma, out, bool(weight_grads), workspace)


# -------------------------------------------- norm and rotation of heads ---

_NORM = {"none": 0, "rms": 1, "layer": 2}


def _norm(kind):
    return _NORM.get(kind, -1)


def qk_norm_rope_fwd(q, k, positions=None, inv_freq=None, q_norm: str = "rms", k_norm: str = "rms", q_gamma=None, q_beta=None,
                     k_gamma=None, k_beta=None, eps: float = 1e-6, axes=None, start: int = 0, interleaved: bool = False,
                     q_out=None, k_out=None, stream=None):
    """Norm of each head of q [..., heads, dim] and k [..., kv_heads, dim] (or
    None) and their position rotation, in one pass: (yq, yk), of their type.

    q_norm, k_norm: "rms", "layer" or "none"; the weights are float32 or of the
    heads' type, all alike, betas a layer norm's only. Heads may lie anywhere in a wider
    buffer (columns of a fused projection); results are contiguous, or go to q_out
    and k_out, q and k themselves among them.

    Pair i of the 2 len(inv_freq) dimensions from `start` on turns by position *
    inv_freq[i] (float32 or float64): dimensions start + i and start + i +
    len(inv_freq), or with `interleaved` start + 2i and start + 2i + 1.
    positions: int32 or int64, one a token; with `axes` (int32, the axis of
    each pair: time, height, width) [axes, ...]. Without positions nothing turns."""
    if stream is not None:
        return _on(stream, qk_norm_rope_fwd, q, k, positions, inv_freq, q_norm, k_norm, q_gamma, q_beta, k_gamma, k_beta, eps,
                   axes, start, interleaved, q_out, k_out)
    return (_n or _native()).qk_norm_rope_fwd(q, k, positions, inv_freq, axes, start, bool(interleaved), _norm(q_norm),
                                              _norm(k_norm), q_gamma, q_beta, k_gamma, k_beta, eps, q_out, k_out)


def qk_norm_rope_bwd_workspace_size(dim: int) -> int:
    return int(load().ibwd_qk_norm_rope_bwd_workspace_size(dim)) if 0 < dim < 1 << 31 else 0


def qk_norm_rope_bwd(dyq, dyk, q, k, positions=None, inv_freq=None, q_norm: str = "rms", k_norm: str = "rms", q_gamma=None,
                     k_gamma=None, eps: float = 1e-6, axes=None, start: int = 0, interleaved: bool = False, q_out=None,
                     k_out=None, weight_grads: bool = True, workspace=None, stream=None):
    """Backward pass of qk_norm_rope_fwd: (dq, dk, dq_gamma, dq_beta, dk_gamma,
    dk_beta), dq and dk of the heads' type, the weights' float32, each None where
    there is none (betas of a layer norm only; none without `weight_grads`).

    q and k are the forward pass's inputs; dyq and dyk have their type or
    float32 (as indexer_backward gives dq and dk). q_out and k_out may supply dq
    and dk: q and k, or dyq and dyk where the types agree, among them. `workspace`:
    a contiguous tensor of qk_norm_rope_bwd_workspace_size bytes (allocated when not given)."""
    if stream is not None:
        return _on(stream, qk_norm_rope_bwd, dyq, dyk, q, k, positions, inv_freq, q_norm, k_norm, q_gamma, k_gamma, eps, axes,
                   start, interleaved, q_out, k_out, weight_grads, workspace)
    return (_n or _native()).qk_norm_rope_bwd(dyq, dyk, q, k, positions, inv_freq, axes, start, bool(interleaved),
                                              _norm(q_norm), _norm(k_norm), q_gamma, k_gamma, eps, q_out, k_out,
                                              bool(weight_grads), workspace)


# ------------------------------------------------- token log probabilities ---

def token_logprobs_fwd(logits, tokens=None, top_n: int = 0, temperature: float = 1.0, stream=None):
    """Log probabilities of `tokens` (int32, one a row; padding outside the
    vocabulary gives 0), the rows' entropies, their log-sum-exp, and the ids
    (int32) and log probabilities of the top_n largest logits, best first.

    Returns (logprob, entropy, lse, top_ids, top_logprobs); logprob is None
    without tokens, the last two without top_n."""
    if stream is not None:
        return _on(stream, token_logprobs_fwd, logits, tokens, top_n, temperature)
    return (_n or _native()).token_logprobs_fwd(logits, tokens, top_n, temperature)


def token_logprobs_bwd(logits, tokens, lse, entropy=None, dlogprob=None, dentropy=None, temperature: float = 1.0,
                       out=None, stream=None):
    """Gradient of the log probabilities (dlogprob) and the entropies
    (dentropy, which needs entropy) with respect to the logits; `out` may
    supply it, the logits themselves among it."""
    if stream is not None:
        return _on(stream, token_logprobs_bwd, logits, tokens, lse, entropy, dlogprob, dentropy, temperature, out)
    return (_n or _native()).token_logprobs_bwd(logits, tokens, lse, entropy, dlogprob, dentropy, temperature, out)


# ----------------------------------------------------------- distillation ---

def distill_fwd(logits, ids, teacher, temperature: float = 1.0, stream=None):
    """Distillation loss of each row against a teacher's kept tokens: ids
    (int32 [..., K], padding outside the vocabulary) with their logits or log
    probabilities `teacher` (float32).  With p the softmax of teacher / T over
    the kept slots and q that of logits / T over the vocabulary,
    loss = T^2 sum p (log p - log q).  Returns (loss, lse)."""
    if stream is not None:
        return _on(stream, distill_fwd, logits, ids, teacher, temperature)
    return (_n or _native()).distill_fwd(logits, ids, teacher, temperature)


def distill_bwd(logits, ids, teacher, lse, dloss, temperature: float = 1.0, out=None, stream=None):
    """Gradient of distill_fwd's losses with respect to the logits, given the
    losses' own gradient dloss; `out` may supply it, the logits among it."""
    if stream is not None:
        return _on(stream, distill_bwd, logits, ids, teacher, lse, dloss, temperature, out)
    return (_n or _native()).distill_bwd(logits, ids, teacher, lse, dloss, temperature, out)


def distill_grad(logits, ids, teacher, row_weight=None, grad_scale: float = 1.0, temperature: float = 1.0, out=None,
                 stream=None):
    """Loss and gradient in one call: (loss, dlogits) with dlogits the
    gradient of grad_scale * sum row_weight * loss (row_weight float32, one a
    row; None for 1).  `out` may supply dlogits, the logits among it."""
    if stream is not None:
        return _on(stream, distill_grad, logits, ids, teacher, row_weight, grad_scale, temperature, out)
    return (_n or _native()).distill_grad(logits, ids, teacher, row_weight, grad_scale, temperature, out)
