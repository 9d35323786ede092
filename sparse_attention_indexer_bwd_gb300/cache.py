"""The cache that a model with an indexer answers from: keys and values, or an
indexer's keys alone, in 8 bits and pages, and the attention over it (declared
in include/indexer_cache.h; the functions drop the C names' ibwd_).

A cache is a contiguous tensor [pages, heads, page, dim] of float8_e4m3fn or
int8 with a float32 scale [pages, heads] for each block, one head's tokens of a
page. page: 16, 32, 64, 128 or 256; dim: a multiple of 16 up to 512. Zeros are an
empty cache. Sequence b has lens[b] tokens, position t in slot t % page of
page page_table[b, t // page] (int32). Without `cu` a call has one token a
sequence; with cu (int32 [sequences + 1]) sequence b has the packed tokens
cu[b] .. cu[b + 1], its last ones, and those before cu[0] or from cu[-1] on are nobody's. lens counts them: a write and the attention
behind it take the same lens, cu and page_table.

Page numbers, lengths and offsets are data of the device: what lies outside is
no token, and is never followed out of bounds. Streams, errors and argument
checks are those of the training operators (train.py).
"""
from __future__ import annotations

import ctypes

import torch

from . import load, train

_CODE = train._CODE

EXPORTS = (
    "ibwd_cache_write",
    "ibwd_cache_read",
    "ibwd_cache_attention_workspace_size",
    "ibwd_cache_attention",
)


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the functions above."""
    p, i, f, sz, n = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
    lib.ibwd_cache_write.argtypes = [p, n, n, p, n, n, i, p, p, p, p]
    lib.ibwd_cache_read.argtypes = [p, p, p, i, i, p]
    lib.ibwd_cache_attention_workspace_size.argtypes = [i]
    lib.ibwd_cache_attention.argtypes = [p, n, n, i, i, p, p, p, p, i, f, p, p, p, sz, p]
    for name in EXPORTS:
        getattr(lib, name).restype = sz if name.endswith("workspace_size") else i


def cache_write(k, v, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu=None, stream=None) -> None:
    """Writes the packed tokens' keys and values [..., heads, dim] (v, v_cache
    and v_scale None for keys alone) as the last tokens of their sequences.

    A block's scale is the least power of two at which none of its finite values
    is beyond the largest code (448, 127); a token that raises it has the older
    tokens' codes rounded anew, and a page whose slot 0 is written begins anew.
    Infinities become the largest code, as do values beyond 127 * 2^120 in int8;
    NaN stays NaN, in int8 as the block's scale."""
    if stream is not None:
        return train._on(stream, cache_write, k, v, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu)
    (train._n or train._native()).cache_write(k, v, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu)


def cache_read(cache, scale, page_table, lens, length: int, dtype=torch.bfloat16, out=None, stream=None):
    """The sequences' first `length` positions, [sequences, length, heads, dim]
    of `dtype`, 0 behind a sequence's end: of an indexer's keys, with one head,
    squeezed, what indexer_fwd takes. `out` may supply it (then its type counts)."""
    if stream is not None:
        return train._on(stream, cache_read, cache, scale, page_table, lens, length, dtype, out)
    if isinstance(out, torch.Tensor):
        dtype = out.dtype
    code = _CODE.get(dtype, -1)
    if code < 0:
        raise ValueError(f"dtype: expected float32, bfloat16 or float16, got {dtype}")
    return (train._n or train._native()).cache_read(cache, scale, page_table, lens, length, code, out)


def cache_attention_workspace_size(dim: int) -> int:
    return int(load().ibwd_cache_attention_workspace_size(dim)) if 0 < dim < 1 << 31 else 0


def cache_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu=None, select=None, scale=None, workspace=None,
                    out=None, stream=None):
    """Attention of the packed tokens' queries [..., heads, dim] (bfloat16 or
    float16; dim 64, 128 or 256) over the cache, heads a multiple of the cache's:
    (out, lse), out of q's shape and type, lse float32 (natural logarithm).

    A token sees the positions up to its own; with `select` (int32 [..., kept],
    an indexer's choice, padding outside) those of them that its row lists. A token
    that sees nothing has out 0 and lse -inf; rows before cu[0] and from cu[-1] on are left as they
    were (undefined where the call allocates the results). scale: of the logits,
    1 / sqrt(dim) by default. Weights and queries are taken with 11 bits (in float16,
    relative to the largest), sums and the softmax's statistics in float32. `workspace`: a contiguous tensor of
    cache_attention_workspace_size bytes (allocated when not given), of one call
    at a time."""
    if stream is not None:
        return train._on(stream, cache_attention, q, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu, select, scale,
                         workspace, out)
    return (train._n or train._native()).cache_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, cu, select,
                                                         scale, workspace, out)
