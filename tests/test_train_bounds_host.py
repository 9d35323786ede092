"""The bounds of train_tight.py on rows with masked logits and padded slots: the
exact results pass, rounded to fp32, and results with a small mistake do not."""
import math

import pytest
import torch

from train_ref import distill, logp_fwd
from train_tight import tight_distill, tight_distill_grad, tight_logp_bwd, tight_logp_fwd

INF = math.inf


def rows(v, fill, kind=torch.float32):
    g = torch.Generator().manual_seed(v)
    x = torch.randn((5, v), generator=g) * 2.5
    x[:, ::3] = fill
    x[3] = fill
    x[3, 4] = 1.0
    return x.to(kind)


def slots(x, k):
    """The largest logits as a teacher's slots, a third of them padding that holds anything."""
    val, ids = torch.topk(torch.where(x > -1e30, x, -40.0).float(), k, dim=1)
    pad = torch.arange(k)[None, :] % 3 == 1
    return (torch.where(pad, x.shape[1] + 3, ids).to(torch.int32),
            torch.where(pad, torch.tensor([1e30, math.nan]).repeat(k)[:k], val + 0.5 * torch.sin(ids.float())))


def fails(check, *args):
    with pytest.raises(AssertionError):
        check(*args)


@pytest.mark.parametrize("fill", [-INF, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("v,k,tau", [(64, 7, 1.0), (4000, 600, 1.0), (4000, 30, 0.7), (4000, 30, 50.0), (999, 30, 1e-3)])
def test_small_mistakes_are_found(v, k, tau, fill):
    x = rows(v, fill)
    tok = torch.tensor([1, 2, 4, 4, v - 2], dtype=torch.int32)
    ref = logp_fwd(x, tok, 5, tau)
    fine = [t if t.dtype == torch.int32 else t.float() for t in ref]
    tight_logp_fwd(fine, x, tok, 5, tau, "exact")
    for i, off in ((0, 0.01), (1, 0.02), (2, 0.01 + 1e-6 * ref[2].abs().max().item()), (4, 0.01)):
        wrong = list(fine)
        wrong[i] = fine[i] + off * (1 + 1e-4 * fine[i].abs())
        fails(tight_logp_fwd, wrong, x, tok, 5, tau, "off")
    a, h = torch.tensor([1.0, -2.0, 0.5, 1.0, 3.0]), torch.tensor([0.1, 0.2, -0.3, 0.4, 0.5])
    lse, ent = fine[2], fine[1]
    lq = x.double() / tau - lse.double()[:, None]
    q = lq.exp()
    hot = torch.nn.functional.one_hot(tok.long(), v)
    part = h.double()[:, None] * q * (torch.where(q == 0, 0.0, lq) + ent.double()[:, None])
    g = (a.double()[:, None] * (hot - q) - part) / tau
    tight_logp_bwd(g.float(), x, tok, lse, ent, a, h, tau, "exact")
    fails(tight_logp_bwd, (a.double()[:, None] * (hot - q) / tau + 1e-3 * q).float(), x, tok, lse, ent, a, h, tau, "no entropy")
    fails(tight_logp_bwd, (a.double()[:, None] * hot / tau).float(), x, tok, lse, ent, a, h, tau, "no probabilities")
    fails(tight_logp_bwd, (g - a.double()[:, None] * hot / tau).float(), x, tok, lse, ent, a, h, tau, "no token")
    ids, teacher = slots(x, k)
    loss, lse, grad, _, full, _ = distill(x, ids, teacher, tau)
    w = torch.tensor([1.0, 0.5, 2.0, 1.0, 0.25])
    tight_distill(loss.float(), lse.float(), x, ids, teacher, tau, "exact")
    tight_distill_grad((grad * w.double()[:, None]).float(), w, x, ids, teacher, tau, "exact")
    fails(tight_distill, loss.float() * 1.001 + 0.01 * tau * tau, None, x, ids, teacher, tau, "loss")
    fails(tight_distill, None, lse.float() * 1.001 + 0.01, x, ids, teacher, tau, "lse")
    fails(tight_distill_grad, ((grad + tau * full) * w.double()[:, None]).float(), w, x, ids, teacher, tau, "no teacher")
    fails(tight_distill_grad, (-tau * full * w.double()[:, None]).float(), w, x, ids, teacher, tau, "no student")
    fails(tight_distill_grad, (grad * w.double()[:, None] * 1.01).float(), w, x, ids, teacher, tau, "1 % off")
