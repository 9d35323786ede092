"""Refusals of the training operators on device tensors: nothing is launched
and no output is touched."""
import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd

pytestmark = pytest.mark.gpu


def refused(status, call, *args, **kwargs):
    with pytest.raises(ibwd.IndexerBwdError) as e:
        call(*args, **kwargs)
    assert e.value.status == status


def norm_args(n=64, rows=6, dtype=torch.bfloat16):
    x = torch.randn((rows, n), device="cuda").to(dtype)
    return x, torch.ones(n, device="cuda"), torch.zeros(rows, device="cuda")


def test_layer_norm():
    x, w, m = norm_args()
    for bad in (x.t(), x[:, ::2], x[:1].expand(6, 64), x.long(), x[0], x.cpu()):
        with pytest.raises(ValueError):
            ibwd.layer_norm_fwd(bad)
    for bad in (w[:-1], w.half(), w.double(), torch.ones(128, device="cuda")[::2], w.cpu()):
        with pytest.raises(ValueError):
            ibwd.layer_norm_fwd(x, bad)
    with pytest.raises(ValueError):
        ibwd.layer_norm_fwd(x, w, w.bfloat16())
    with pytest.raises(ValueError):
        ibwd.layer_norm_fwd(x, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        ibwd.layer_norm_fwd(x, out=torch.empty_like(x[:-1]))
    out = torch.full_like(x, 7)
    for eps in (-1.0, float("nan"), float("inf")):
        refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.layer_norm_fwd, x, eps=eps, out=out)
    refused(ibwd.IBWD_ERR_UNSUPPORTED, ibwd.layer_norm_fwd, x, out_dtype=torch.float32)
    assert (out == 7).all()
    for bad in (m[:-1], m.double(), m.cpu(), m[:, None]):
        with pytest.raises(ValueError):
            ibwd.layer_norm_bwd(x, x, bad, m)
        with pytest.raises(ValueError):
            ibwd.layer_norm_bwd(x, x, m, bad)
    with pytest.raises(ValueError):
        ibwd.layer_norm_bwd(x[:-1], x, m, m)
    refused(ibwd.IBWD_ERR_UNSUPPORTED, ibwd.layer_norm_bwd, x.half(), x, m, m)
    small = torch.empty(16, device="cuda", dtype=torch.uint8)
    refused(ibwd.IBWD_ERR_WORKSPACE, ibwd.layer_norm_bwd, x, x, m, m, out=out, workspace=small)
    refused(ibwd.IBWD_ERR_WORKSPACE, ibwd.layer_norm_bwd, x, x, m, m, out=out,
            workspace=torch.empty(1 << 20, dtype=torch.uint8))
    assert (out == 7).all()
    # in place, but with another row stride
    wide = torch.zeros((6, 80), device="cuda", dtype=torch.bfloat16)
    y = wide.as_strided((6, 64), (64, 1))
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.layer_norm_fwd, wide[:, :64], out=y)


def test_logits():
    x = torch.randn((4, 100), device="cuda")
    tok = torch.zeros(4, device="cuda", dtype=torch.int32)
    f = torch.zeros(4, device="cuda")
    for bad in (tok.long(), tok[:-1], tok.cpu(), tok[:, None]):
        with pytest.raises(ValueError):
            ibwd.token_logprobs_fwd(x, bad)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.token_logprobs_fwd, x, tok, top_n=101)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.token_logprobs_fwd, x, tok, top_n=-1)
    refused(ibwd.IBWD_ERR_UNSUPPORTED, ibwd.token_logprobs_fwd, torch.randn((2, 300), device="cuda"), None, top_n=129)
    out = torch.full_like(x, 7)
    ids = torch.zeros((4, 3), device="cuda", dtype=torch.int32)
    teacher = torch.zeros((4, 3), device="cuda")
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.token_logprobs_fwd, x, tok, temperature=tau)
        refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.token_logprobs_bwd, x, tok, f, f, f, f, temperature=tau, out=out)
        refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.distill_fwd, x, ids, teacher, temperature=tau)
        refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.distill_bwd, x, ids, teacher, f, f, temperature=tau, out=out)
        refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.distill_grad, x, ids, teacher, temperature=tau, out=out)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.token_logprobs_bwd, x, None, f, None, None, f, out=out)  # needs entropy
    with pytest.raises(TypeError):
        ibwd.token_logprobs_bwd(x, tok, None)
    with pytest.raises(ValueError):
        ibwd.token_logprobs_bwd(x, tok, f, f, f, f, out=out.half())
    for bad in (ids.long(), ids[:, :0], ids[:-1], ids[0], ids.cpu()):
        with pytest.raises((ValueError, ibwd.IndexerBwdError)):
            ibwd.distill_grad(x, bad, teacher[:, :0] if bad.dim() == 2 and bad.shape[1] == 0 else teacher, out=out)
    for bad in (teacher.half(), teacher[:, :2], teacher.t()):
        with pytest.raises(ValueError):
            ibwd.distill_grad(x, ids, bad, out=out)
    wide = torch.zeros((4, 1025), device="cuda")
    refused(ibwd.IBWD_ERR_UNSUPPORTED, ibwd.distill_grad, x, wide.int(), wide, out=out)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.distill_grad, x, ids, teacher, grad_scale=float("nan"), out=out)
    with pytest.raises(ValueError):
        ibwd.distill_grad(x, ids, teacher, row_weight=f[:-1], out=out)
    assert (out == 7).all()
    assert ibwd.indexer_bwd_last_device_status() == ibwd.IBWD_OK
