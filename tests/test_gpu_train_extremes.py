"""Values at the ends of the types' ranges, and NaN, where a result still has one value."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd

pytestmark = pytest.mark.gpu

INF = math.inf
SHAPES = [(3, 40000), (320, 1504)]


@pytest.mark.parametrize("tau", [1.0, 4.0])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_gradients_of_a_row_of_the_lowest_value(kind, tau):
    """log p = x / T - lse is 0 in fp32 for every token of such a row: p = 1, by the lse that the forward pass can give."""
    for rows, v in SHAPES:
        x = torch.full((rows, v), torch.finfo(kind).min, device="cuda", dtype=kind)
        tok = torch.full((rows,), 5, device="cuda", dtype=torch.int32)
        _, entropy, lse, _, _ = ibwd.token_logprobs_fwd(x, tok, temperature=tau)
        assert torch.isfinite(lse).all()
        one = torch.ones(rows, device="cuda")
        dx = ibwd.token_logprobs_bwd(x, tok, lse, entropy, one, None, temperature=tau).float()
        assert (dx[:, 5] == 0).all() and (dx[:, 6:] + 1 / tau).abs().max() < 0.01
        ids, teacher = tok[:, None].contiguous(), one[:, None].contiguous()
        _, lse = ibwd.distill_fwd(x, ids, teacher, temperature=tau)
        dx = ibwd.distill_bwd(x, ids, teacher, lse, one, temperature=tau).float()
        assert (dx[:, 5] == 0).all() and (dx[:, 6:] - tau).abs().max() < 0.02 * tau


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_a_logit_near_the_largest_value(kind):
    """Such a token has all of the probability: entropy 0, and a gradient that is 0 beside it."""
    for rows, v in SHAPES:
        x = torch.randn((rows, v), device="cuda").to(kind)
        x[:, 7] = 3e38
        tok = torch.full((rows,), 7, device="cuda", dtype=torch.int32)
        logprob, entropy, lse, ids, _ = ibwd.token_logprobs_fwd(x, tok, top_n=2)
        assert (logprob == 0).all() and (entropy == 0).all() and (lse == x[:, 7].float()).all() and (ids[:, 0] == 7).all()
        one = torch.ones(rows, device="cuda")
        assert (ibwd.token_logprobs_bwd(x, tok, lse, entropy, one, one) == 0).all()
        kept = tok[:, None].contiguous()
        loss, dx = ibwd.distill_grad(x, kept, one[:, None].contiguous())
        assert (loss == 0).all() and (dx == 0).all()
        loss, lse = ibwd.distill_fwd(x, kept, one[:, None].contiguous())
        assert (loss == 0).all()
        assert (ibwd.distill_bwd(x, kept, one[:, None].contiguous(), lse, one) == 0).all()


def test_mean_of_a_row_with_an_infinity():
    """Sum / N is that infinity, at every width."""
    for n in (8, 100, 512, 2047, 4096, 9001, 16384, 20000):
        for kind in (torch.bfloat16, torch.float32):
            x = torch.randn((12, n), device="cuda").to(kind)
            x[3, n // 2] = INF
            x[4, 0] = -INF
            x[5, 1], x[5, 3] = INF, -INF
            mean = ibwd.layer_norm_fwd(x)[1]
            assert mean[3] == INF and mean[4] == -INF and torch.isnan(mean[5]), n


def test_nan_among_the_teacher():
    """A kept slot's NaN is the loss's, whatever the other slots hold; a padding slot's is not."""
    for rows, v in SHAPES:
        x = torch.randn((rows, v), device="cuda")
        ids = torch.arange(4, device="cuda", dtype=torch.int32).expand(rows, 4).contiguous()
        teacher = torch.zeros((rows, 4), device="cuda")
        teacher[0] = torch.tensor([math.nan, -INF, -INF, -INF])
        teacher[1, 2] = math.nan
        teacher[2] = -math.nan
        ids[2, 1:] = -1
        other = [i for i in range(rows) if i > 2]
        for k in (1, 2, 4):
            loss = [ibwd.distill_grad(x, ids[:, :k].contiguous(), teacher[:, :k].contiguous())[0],
                    ibwd.distill_fwd(x, ids[:, :k].contiguous(), teacher[:, :k].contiguous())[0]]
            for got in loss:
                assert torch.isnan(got[0]) and torch.isnan(got[1]) == (k > 2) and torch.isnan(got[2])
                assert torch.isfinite(got[other]).all()
        teacher[:3] = math.nan
        ids[:3] = -1
        ids[:3, 3] = 9
        teacher[:3, 3] = 0
        for got in (ibwd.distill_grad(x, ids, teacher)[0], ibwd.distill_fwd(x, ids, teacher)[0]):
            assert torch.isfinite(got).all()


@pytest.mark.parametrize("tau", [1.0, 0.7, 0.01])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_several_kept_tokens_that_the_student_masks_by_the_lowest_value(kind, tau):
    """The loss is T times the mean of what they cost, about the largest value itself and no infinity."""
    low = torch.finfo(kind).min
    for rows, v in SHAPES:
        x = torch.randn((rows, v), device="cuda").to(kind)
        ids = torch.arange(40, 104, device="cuda", dtype=torch.int32).expand(rows, 64).contiguous()
        x[:, 40:104] = low
        x[:, 48] = 1
        teacher = torch.zeros((rows, 64), device="cuda")
        want = -low * 63 / 64 * tau
        for call in (ibwd.distill_grad, ibwd.distill_fwd):
            got = call(x, ids, teacher, temperature=tau)[0]
            assert ((got.double() - want).abs() <= 1e-5 * want).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
def test_top_of_a_row_with_vectors_of_nan(kind):
    """NaN is no alternative: the ids are those of the largest other logits."""
    for rows, v in ((2, 2048), (400, 2048), (2, 20000)):
        x = torch.full((rows, v), -1000.0, device="cuda")
        x[:, 11] = 5  # far above all others: the bound is searched for
        x += torch.arange(v, device="cuda") % 97
        for y in (x, x - 16, -(torch.arange(v, device="cuda") % 97).expand(rows, v) - 1e-3):  # (the last: all but 0)
            y = y.to(kind)
            y[:, v // 4:3 * v // 4] = math.nan
            for n in (1, 64, 128):
                got = ibwd.token_logprobs_fwd(y, None, top_n=n)[3]
                key = torch.where(torch.isnan(y), -INF, y.double())
                want = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :n]
                assert torch.equal(got.long(), want), (rows, v, n)


def test_nan_stays_in_its_row():
    """Every operator over logits, forward and backward: NaN in one row's logits or statistics and in no other's."""
    for rows, v in SHAPES:
        x = torch.randn((rows, v), device="cuda")
        tok = torch.full((rows,), 3, device="cuda", dtype=torch.int32)
        ids = torch.arange(4, device="cuda", dtype=torch.int32).expand(rows, 4).contiguous()
        teacher, one = torch.zeros((rows, 4), device="cuda"), torch.ones(rows, device="cuda")

        def all_of(x):
            logprob, entropy, lse, _, best = ibwd.token_logprobs_fwd(x, tok, top_n=3)
            loss, lse2 = ibwd.distill_fwd(x, ids, teacher)
            whole, dw = ibwd.distill_grad(x, ids, teacher)
            return (logprob, entropy, lse, best, ibwd.token_logprobs_bwd(x, tok, lse, entropy, one, one), loss, lse2,
                    ibwd.distill_bwd(x, ids, teacher, lse2, one), whole, dw)

        clean = all_of(x)
        y = x.clone()
        y[1, v // 3] = math.nan
        y[1, 5] = -INF
        for a, b in zip(all_of(y), clean):
            assert torch.isnan(a[1]).all()
            assert torch.equal(a[0], b[0]) and torch.equal(a[2:], b[2:])
