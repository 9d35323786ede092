"""Refusals of the norm and rotation of heads, the 8-bit cache and its attention without a GPU: the library's checks
before any launch, and the binding's of host tensors."""
import ctypes
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd

P = 4096  # never dereferenced: the checks under test come first
INVALID, UNSUPPORTED, WORKSPACE = ibwd.IBWD_ERR_INVALID_ARG, ibwd.IBWD_ERR_UNSUPPORTED, ibwd.IBWD_ERR_WORKSPACE
i64, i32, ptr = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p


class Heads(ctypes.Structure):
    _fields_ = [("x", ptr), ("x_token", i64), ("x_head", i64), ("heads", i32), ("norm", i32), ("gamma", ptr), ("beta", ptr),
                ("y", ptr), ("y_token", i64), ("y_head", i64), ("dy", ptr), ("dy_type", i32), ("dy_token", i64),
                ("dy_head", i64), ("dgamma", ptr), ("dbeta", ptr)]


class Rotation(ctypes.Structure):
    _fields_ = [("positions", ptr), ("positions_int64", i32), ("axis_stride", i64), ("axes", i32), ("axis_of", ptr),
                ("freq", ptr), ("freq_f64", i32), ("pairs", i32), ("start", i32), ("interleaved", i32)]


class Cache(ctypes.Structure):
    _fields_ = [("codes", ptr), ("scale", ptr)]


class Sequences(ctypes.Structure):
    _fields_ = [("table", ptr), ("table_stride", i64), ("table_width", i32), ("batch", i32), ("lens", ptr), ("cu", ptr),
                ("tokens", i64), ("pages", i64), ("heads", i32), ("page", i32), ("dim", i32), ("code", i32)]


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_bwd_gb300 import _build
    _build.build()
    return ibwd.load()


def heads(**kw):
    d = dict(x=P, x_token=256, x_head=64, heads=4, norm=1, gamma=P, beta=None, y=8 * P, y_token=256, y_head=64, dy=16 * P,
             dy_type=1, dy_token=256, dy_head=64, dgamma=P, dbeta=None)
    return Heads(**{**d, **kw})


def rotation(**kw):
    d = dict(positions=P, positions_int64=0, axis_stride=8, axes=1, axis_of=None, freq=P, freq_f64=1, pairs=32, start=0,
             interleaved=0)
    return Rotation(**{**d, **kw})


def fwd(lib, q=None, k=None, r=None, type_=1, w=0, tokens=8, dim=64, eps=1e-6):
    q = q or heads()
    return lib.ibwd_qk_norm_rope_fwd(ctypes.byref(q), ctypes.byref(k) if k else None, ctypes.byref(r or rotation()), type_, w,
                                     tokens, dim, eps, None)


def bwd(lib, q=None, k=None, r=None, type_=1, w=0, tokens=8, dim=64, eps=1e-6, ws=P, size=1 << 20):
    q = q or heads()
    return lib.ibwd_qk_norm_rope_bwd(ctypes.byref(q), ctypes.byref(k) if k else None, ctypes.byref(r or rotation()), type_, w,
                                     tokens, dim, eps, ws, size, None)


def test_norm_and_rotation(lib):
    for call in (fwd, bwd):
        assert call(lib, tokens=-1) == INVALID
        assert call(lib, dim=0) == INVALID
        assert call(lib, dim=513) == UNSUPPORTED
        assert call(lib, type_=3) == INVALID
        assert call(lib, type_=1, w=2) == UNSUPPORTED
        assert call(lib, tokens=(1 << 27) + 1) == UNSUPPORTED
        for eps in (-1e-9, math.nan, math.inf):
            assert call(lib, eps=eps) == INVALID
        for bad in (dict(heads=-1), dict(norm=3), dict(norm=0), dict(y=None), dict(y=8 * P + 1), dict(x_token=-1), dict(x_head=-1),
                    dict(x=P, y=P, y_token=512), dict(y_token=0), dict(y_head=63), dict(y_token=100), dict(gamma=P + 1)):
            assert call(lib, q=heads(**bad)) == INVALID, bad
            assert call(lib, q=heads(), k=heads(**bad)) == INVALID, bad
        assert call(lib, q=heads(x=None)) == INVALID
        assert call(lib, q=heads(heads=(1 << 16) + 1)) == UNSUPPORTED
        assert call(lib, q=heads(x_token=1 << 58)) == UNSUPPORTED
        for bad in (dict(pairs=-1), dict(pairs=33), dict(start=1), dict(start=-2), dict(axes=0), dict(axes=2, axis_stride=7),
                    dict(freq=None), dict(positions=P + 2), dict(freq=P + 4), dict(axis_of=P + 1),
                    dict(positions=P + 4, positions_int64=1)):
            assert call(lib, r=rotation(**bad)) == INVALID, bad
        assert call(lib, r=rotation(axes=9)) == UNSUPPORTED
    assert fwd(lib, q=heads(beta=P)) == INVALID           # a layer norm's only
    assert bwd(lib, q=heads(dy=None)) == INVALID
    assert bwd(lib, q=heads(dy_type=2)) == UNSUPPORTED
    assert bwd(lib, q=heads(dy_type=5)) == INVALID
    assert bwd(lib, q=heads(dy_head=-64)) == INVALID
    assert bwd(lib, q=heads(norm=0, gamma=None)) == INVALID    # sums without a norm
    assert bwd(lib, q=heads(y=16 * P, dy_token=512)) == INVALID
    assert bwd(lib, q=heads(y=16 * P, dy_type=0)) == INVALID
    # a result that is the other operand's result or argument
    for q, k in ((dict(), dict()), (dict(), dict(y=P, x=64 * P)), (dict(y=64 * P), dict(x=64 * P)), (dict(x=64 * P), dict(y=64 * P))):
        for call in (fwd, bwd):
            assert call(lib, q=heads(**q), k=heads(**{"dgamma": 2 * P, **k})) == INVALID, (q, k)
    assert bwd(lib, q=heads(y=64 * P), k=heads(dy=64 * P, dgamma=2 * P)) == INVALID
    assert bwd(lib, q=heads(), k=heads(y=32 * P, dy=64 * P)) == INVALID  # one dgamma for both
    assert bwd(lib, q=heads(norm=2, dbeta=P)) == INVALID
    assert bwd(lib, q=heads(dbeta=2 * P)) == INVALID           # a layer norm's only
    assert bwd(lib, ws=None) == WORKSPACE
    assert bwd(lib, ws=P + 8) == WORKSPACE
    assert fwd(lib, tokens=0) == ibwd.IBWD_OK
    assert bwd(lib, q=heads(dgamma=None), tokens=0) == ibwd.IBWD_OK
    assert ibwd.qk_norm_rope_bwd_workspace_size(128) >= 2 * 128 * 4
    assert ibwd.qk_norm_rope_bwd_workspace_size(0) == ibwd.qk_norm_rope_bwd_workspace_size(513) == 0
    assert ibwd.qk_norm_rope_bwd_workspace_size(1 << 40) == 0


def seqs(**kw):
    d = dict(table=P, table_stride=4, table_width=4, batch=3, lens=P, cu=None, tokens=3, pages=10, heads=2, page=16, dim=64, code=0)
    return Sequences(**{**d, **kw})


def write(lib, s=None, k=P, v=2 * P, type_=1, kc=None, vc=None, token=128, head=64):
    kc, vc = kc or Cache(3 * P, 4 * P), vc if vc is not None else Cache(5 * P, 6 * P)
    return lib.ibwd_cache_write(k, token, head, v, token, head, type_, ctypes.byref(kc), ctypes.byref(vc) if vc else None,
                                ctypes.byref(s or seqs()), None)


def read(lib, s=None, c=None, out=P, type_=1, length=10):
    return lib.ibwd_cache_read(ctypes.byref(c or Cache(3 * P, 4 * P)), ctypes.byref(s or seqs()), out, type_, length, None)


def attend(lib, s=None, q=P, type_=1, group=4, kc=None, vc=None, select=None, kept=0, scale=0.1, out=7 * P, ws=8 * P, size=1 << 30,
           token=512, head=64):
    return lib.ibwd_cache_attention(q, token, head, type_, group, ctypes.byref(kc or Cache(3 * P, 4 * P)),
                                    ctypes.byref(vc or Cache(5 * P, 6 * P)), ctypes.byref(s or seqs()), select, kept, scale, out,
                                    None, ws, size, None)


def test_cache(lib):
    for call in (write, read, attend):
        for bad in (dict(batch=-1), dict(table_width=0), dict(table_stride=3), dict(pages=0), dict(heads=0), dict(dim=0),
                    dict(page=0), dict(tokens=-1), dict(code=2), dict(table=None), dict(lens=None), dict(table=P + 1)):
            assert call(lib, s=seqs(**bad)) == INVALID, (call, bad)
        for bad in (dict(page=8), dict(page=48), dict(page=512), dict(dim=72), dict(dim=528), dict(heads=65536), dict(batch=(1 << 20) + 1),
                    dict(tokens=(1 << 27) + 1), dict(pages=1 << 31), dict(table_width=1 << 30, table_stride=1 << 30)):
            assert call(lib, s=seqs(**bad)) == UNSUPPORTED, (call, bad)
        assert call(lib, type_=4) == INVALID
        assert call(lib, s=seqs(batch=0, tokens=0)) == ibwd.IBWD_OK
    for call in (write, attend):
        assert call(lib, s=seqs(tokens=4)) == INVALID      # without offsets one token a sequence
        assert call(lib, s=seqs(cu=P + 2)) == INVALID
        assert call(lib, token=-1) == INVALID and call(lib, head=-1) == INVALID
        assert call(lib, token=1 << 60) == UNSUPPORTED
        assert call(lib, kc=Cache(3 * P + 8, 4 * P)) == INVALID
        assert call(lib, vc=Cache(5 * P, 6 * P + 2)) == INVALID
        assert call(lib, kc=Cache(None, 4 * P)) == INVALID
        assert call(lib, s=seqs(cu=P, tokens=0)) == ibwd.IBWD_OK
    assert write(lib, k=None) == INVALID and write(lib, k=P + 1) == INVALID
    assert write(lib, v=None) == INVALID and write(lib, vc=False) == INVALID
    assert write(lib, vc=Cache(3 * P, 6 * P)) == INVALID and write(lib, vc=Cache(5 * P, 4 * P)) == INVALID
    assert read(lib, length=-1) == INVALID and read(lib, out=None) == INVALID and read(lib, out=P + 8) == INVALID
    assert read(lib, length=(1 << 31) - 5) == UNSUPPORTED
    assert read(lib, length=1 << 30, s=seqs(batch=1 << 20)) == UNSUPPORTED
    assert read(lib, length=0) == ibwd.IBWD_OK
    assert attend(lib, type_=0) == UNSUPPORTED and attend(lib, s=seqs(dim=80)) == UNSUPPORTED
    assert attend(lib, group=0) == INVALID and attend(lib, group=65536) == UNSUPPORTED
    assert attend(lib, s=seqs(tokens=1 << 20, batch=1 << 20), group=1 << 11) == UNSUPPORTED     # more rows than are counted
    assert attend(lib, s=seqs(cu=P, tokens=1 << 24, heads=1 << 12, table_width=1 << 26, table_stride=1 << 26)) == UNSUPPORTED
    for scale in (math.nan, math.inf, 3e38):
        assert attend(lib, scale=scale) == INVALID
    assert attend(lib, select=P, kept=0) == INVALID and attend(lib, select=P + 1, kept=4) == INVALID
    assert attend(lib, q=None) == INVALID and attend(lib, q=P + 1) == INVALID and attend(lib, out=7 * P + 8) == INVALID
    assert attend(lib, q=7 * P) == INVALID
    assert attend(lib, ws=None) == WORKSPACE and attend(lib, ws=8 * P + 4) == WORKSPACE and attend(lib, size=1000) == WORKSPACE
    for dim in (64, 128, 256):
        assert ibwd.cache_attention_workspace_size(dim) > 0
    for dim in (0, -64, 80, 512, 1 << 40):
        assert ibwd.cache_attention_workspace_size(dim) == 0


def test_host_tensors_and_other_arguments_are_refused(lib):
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cache, scale = torch.zeros((3, 2, 16, 64), dtype=torch.int8), torch.zeros((3, 2))
    table, lens = torch.zeros((4, 1), dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ibwd.qk_norm_rope_fwd(q, q)
    with pytest.raises(ValueError):
        ibwd.qk_norm_rope_bwd(q, q, q, q)
    with pytest.raises(TypeError):
        ibwd.qk_norm_rope_fwd(None, q)
    with pytest.raises(ValueError):
        ibwd.cache_write(q, q, cache, cache, scale, scale, table, lens)
    with pytest.raises(ValueError):
        ibwd.cache_read(cache, scale, table, lens, 4)
    with pytest.raises(ValueError):
        ibwd.cache_read(cache, scale, table, lens, 4, dtype=torch.float64)
    with pytest.raises(ValueError):
        ibwd.cache_attention(q, cache, cache, scale, scale, table, lens)
    with pytest.raises(TypeError):
        ibwd.cache_attention(q, None, cache, scale, scale, table, lens)
