"""Refusals of the training operators without a GPU: the binding's checks of
host tensors, types and shapes, and the library's checks before any launch."""
import ctypes

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd

P = ctypes.c_void_p(4096)  # never dereferenced: the checks under test come first
NAN, INF = float("nan"), float("inf")
INVALID, UNSUPPORTED, WORKSPACE = ibwd.IBWD_ERR_INVALID_ARG, ibwd.IBWD_ERR_UNSUPPORTED, ibwd.IBWD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_bwd_gb300 import _build
    _build.build()
    return ibwd.load()


def norm_fwd(lib, x=P, xt=0, xs=8, g=P, b=P, wt=0, y=ctypes.c_void_p(8192), yt=0, ys=8, rows=2, n=8, eps=1e-5):
    return lib.ibwd_layer_norm_fwd(x, xt, xs, g, b, wt, y, yt, ys, P, P, rows, n, eps, None)


def norm_bwd(lib, dy=P, dyt=0, dys=8, x=P, xt=0, xs=8, wt=0, dx=ctypes.c_void_p(8192), dxs=8, rows=2, n=8, mean=P,
             ws=P, bytes_=1 << 20):
    return lib.ibwd_layer_norm_bwd(dy, dyt, dys, x, xt, xs, P, wt, mean, P, dx, dxs, P, P, rows, n, ws, bytes_, None)


def logp_fwd(lib, x=P, t=0, s=100, tok=P, tau=1.0, lp=P, ids=P, top=P, n=4, rows=2, v=100):
    return lib.ibwd_token_logprobs_fwd(x, t, s, tok, tau, lp, P, P, ids, top, n, rows, v, None)


def logp_bwd(lib, x=P, t=0, s=100, tok=P, tau=1.0, lse=P, ent=P, da=P, dh=P, dx=ctypes.c_void_p(1 << 20), ds=100,
             rows=2, v=100):
    return lib.ibwd_token_logprobs_bwd(x, t, s, tok, tau, lse, ent, da, dh, dx, ds, rows, v, None)


def distill_grad(lib, x=P, t=0, s=100, ids=P, teacher=P, k=4, tau=1.0, scale=1.0, dx=ctypes.c_void_p(1 << 20), ds=100,
                 rows=2, v=100):
    return lib.ibwd_distill_grad(x, t, s, ids, teacher, k, tau, P, scale, P, dx, ds, rows, v, None)


def test_shapes_types_and_values_are_refused(lib):
    for call in (norm_fwd, norm_bwd):
        assert call(lib, rows=-1) == INVALID
        assert call(lib, n=0) == INVALID
        assert call(lib, xs=7) == INVALID
        assert call(lib, xt=3) == INVALID
        assert call(lib, x=None) == INVALID
        assert call(lib, x=ctypes.c_void_p(4097)) == INVALID
        assert call(lib, xt=1, wt=2) == UNSUPPORTED
        assert call(lib, rows=(1 << 27) + 1) == UNSUPPORTED
    assert norm_fwd(lib, xt=1, yt=2) == UNSUPPORTED
    assert norm_fwd(lib, xt=1, yt=0) == UNSUPPORTED
    for eps in (-1e-9, NAN, INF):
        assert norm_fwd(lib, eps=eps) == INVALID
    assert norm_fwd(lib, y=P, ys=9) == INVALID           # in place needs x's stride
    assert norm_fwd(lib, y=P, yt=1) == INVALID           # and x's type
    assert norm_bwd(lib, xt=1, dyt=2) == UNSUPPORTED
    assert norm_bwd(lib, dx=P, dxs=9) == INVALID
    assert norm_bwd(lib, mean=None) == INVALID
    assert norm_bwd(lib, ws=None) == WORKSPACE
    assert norm_bwd(lib, ws=ctypes.c_void_p(4100)) == WORKSPACE
    for call in (logp_fwd, logp_bwd, distill_grad):
        assert call(lib, v=0) == INVALID
        assert call(lib, s=99) == INVALID
        assert call(lib, t=-1) == INVALID
        assert call(lib, x=None) == INVALID
        assert call(lib, v=(1 << 30) + 1, s=1 << 31) == UNSUPPORTED
        for tau in (0.0, -1.0, NAN, INF, 1e-45):
            assert call(lib, tau=tau) == INVALID
    assert logp_fwd(lib, n=-1) == INVALID
    assert logp_fwd(lib, n=101) == INVALID
    assert logp_fwd(lib, v=200, s=200, n=129) == UNSUPPORTED
    assert logp_fwd(lib, n=0) == INVALID                 # buffers without alternatives
    assert logp_fwd(lib, ids=None) == INVALID
    assert logp_fwd(lib, tok=None) == INVALID            # logprob without tokens
    assert logp_bwd(lib, tok=None) == INVALID
    assert logp_bwd(lib, ent=None) == INVALID
    assert logp_bwd(lib, lse=None) == INVALID
    for call in (logp_bwd, distill_grad):
        assert call(lib, ds=99) == INVALID
        assert call(lib, dx=P, ds=101) == INVALID
        assert call(lib, dx=None) == INVALID
    assert distill_grad(lib, k=0) == INVALID
    assert distill_grad(lib, k=1025) == UNSUPPORTED
    assert distill_grad(lib, ids=None) == INVALID
    for scale in (NAN, INF):
        assert distill_grad(lib, scale=scale) == INVALID


def test_no_rows_need_no_device(lib):
    assert norm_fwd(lib, rows=0) == ibwd.IBWD_OK
    assert logp_fwd(lib, rows=0) == ibwd.IBWD_OK
    assert logp_bwd(lib, rows=0) == ibwd.IBWD_OK
    assert distill_grad(lib, rows=0) == ibwd.IBWD_OK


def test_workspace_size(lib):
    assert ibwd.layer_norm_bwd_workspace_size(0, 128) > 0
    assert ibwd.layer_norm_bwd_workspace_size(4096, 128) >= 2 * 128 * 4
    assert ibwd.layer_norm_bwd_workspace_size(-1, 128) == 0
    assert ibwd.layer_norm_bwd_workspace_size(4, 0) == 0


def test_host_tensors_and_other_types_are_refused(lib):
    x = torch.zeros((4, 16))
    with pytest.raises(ValueError):
        ibwd.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        ibwd.layer_norm_bwd(x, x, x[:, 0], x[:, 0])
    with pytest.raises(ValueError):
        ibwd.token_logprobs_fwd(x, None)
    with pytest.raises(ValueError):
        ibwd.token_logprobs_bwd(x, None, x[:, 0])
    for f in (ibwd.distill_fwd, ibwd.distill_grad):
        with pytest.raises(ValueError):
            f(x, x[:, :2].int(), x[:, :2])
    with pytest.raises(TypeError):
        ibwd.layer_norm_fwd(None)
    with pytest.raises(TypeError):
        ibwd.token_logprobs_fwd([1.0])
