"""The tensors that the training operators give back: their layout, and their versions."""
import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd

pytestmark = pytest.mark.gpu


def size_of(t):
    return t.untyped_storage().nbytes()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_results_of_a_slice_do_not_keep_its_gaps(kind):
    wide = torch.randn((3, 50, 4096), device="cuda").to(kind)
    x = wide[..., 512:512 + 128]
    y, mean, rstd = ibwd.layer_norm_fwd(x)
    dx, dg, db = ibwd.layer_norm_bwd(x, x, mean, rstd)
    _, entropy, lse, _, _ = ibwd.token_logprobs_fwd(x)
    dl = ibwd.token_logprobs_bwd(x, None, lse, entropy, None, lse)
    ids = torch.zeros((3, 50, 2), device="cuda", dtype=torch.int32)
    teacher = torch.zeros((3, 50, 2), device="cuda")
    db = ibwd.distill_bwd(x, ids, teacher, lse, lse)
    dd = ibwd.distill_grad(x, ids, teacher)[1]
    same = ibwd.layer_norm_fwd(x.contiguous())[0]
    for t in (y, dx, dl, db, dd):
        assert t.is_contiguous() and t.shape == x.shape and t.dtype == kind
    assert torch.equal(y, same)


@pytest.mark.parametrize("n,first,pitch", [(127, 0, 4096), (127, 3, 4099), (1001, 1, 50000), (100, 8, 3001), (1, 5, 700)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_results_of_odd_slices_are_small(kind, n, first, pitch):
    """Rows that begin anywhere: a result's rows are at most a cache line longer than what they hold."""
    x = torch.randn((40, pitch), device="cuda").to(kind)[:, first:first + n]
    y, mean, rstd = ibwd.layer_norm_fwd(x)
    dx = ibwd.layer_norm_bwd(x, x, mean, rstd)[0]
    for t in (y, dx):
        assert t.shape == x.shape and t.stride(1) == 1 and t.stride(0) < n + 128 // t.element_size()
        assert size_of(t) <= 2 * 512 + 40 * (n * t.element_size() + 128)
    assert (y.float() - ibwd.layer_norm_fwd(x.contiguous())[0].float()).abs().max() < 0.05


def test_keys_of_a_fused_projection():
    """Keys that are some columns of a wider product go through the norm to the indexer and back."""
    B, S, H, D, L = 2, 64, 8, 128, 32
    g = torch.Generator(device="cuda").manual_seed(0)
    fused = torch.randn((B, S, D + H + 1024), device="cuda", generator=g).bfloat16()
    q = torch.randn((B, S, H, D), device="cuda", generator=g).bfloat16()
    w = torch.randn((B, S, H), device="cuda", generator=g)
    idx = torch.arange(L, device="cuda", dtype=torch.int32).expand(B, S, L).contiguous()
    idx = torch.where(idx <= torch.arange(S, device="cuda")[None, :, None], idx, -1).to(torch.int32)
    raw = fused[..., :D]
    k, mean, rstd = ibwd.layer_norm_fwd(raw, eps=1e-6)
    scores = ibwd.indexer_fwd(q, k, w, idx)
    k2 = ibwd.layer_norm_fwd(raw.contiguous(), eps=1e-6)[0]
    assert torch.equal(scores, ibwd.indexer_fwd(q, k2, w, idx))
    target = torch.softmax(torch.where(idx >= 0, torch.zeros_like(scores), -torch.inf), -1)
    _, _, dk = ibwd.indexer_backward(q, k, w, scores, target, idx)
    draw, _, _ = ibwd.layer_norm_bwd(dk, raw, mean, rstd)
    assert draw.is_contiguous() and torch.isfinite(draw).all()


def test_a_tensor_written_as_out_has_a_new_version():
    """What autograd saved before it was overwritten is found out by its version."""
    x = torch.randn((4, 64), device="cuda")
    ids = torch.zeros((4, 2), device="cuda", dtype=torch.int32)
    teacher = torch.zeros((4, 2), device="cuda")
    _, mean, rstd = ibwd.layer_norm_fwd(x)
    _, entropy, lse, _, _ = ibwd.token_logprobs_fwd(x)
    out = torch.empty_like(x)
    before = x._version
    for call in (lambda: ibwd.layer_norm_fwd(x, out=out), lambda: ibwd.layer_norm_bwd(x, x, mean, rstd, out=out),
                 lambda: ibwd.token_logprobs_bwd(x, None, lse, entropy, None, lse, out=out),
                 lambda: ibwd.distill_bwd(x, ids, teacher, lse, lse, out=out),
                 lambda: ibwd.distill_grad(x, ids, teacher, out=out)):
        at = out._version
        call()
        assert out._version > at
    assert x._version == before
    with torch.inference_mode():
        y = torch.empty_like(x)
    ibwd.layer_norm_fwd(x, out=y)
    a = torch.randn((4, 64), device="cuda", requires_grad=True)
    b = a * 2
    loss = (b * b).sum()  # saves b
    ibwd.layer_norm_fwd(b.detach(), out=b.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
