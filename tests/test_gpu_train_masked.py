"""Operators over logits on rows with masked logits, padded slots and extreme
temperatures, within bounds that such rows leave small (train_tight.py)."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from test_gpu_train_logits import logits, some_tokens
from train_ref import DTYPES
from train_tight import tight_distill, tight_distill_grad, tight_logp_bwd, tight_logp_fwd

pytestmark = pytest.mark.gpu

INF = math.inf


def teacher_of(x, k, seed=2):
    """The student's largest logits moved by noise; a fifth of the slots is padding that holds NaN or 1e30."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.where(x.float() > -60000, x.float(), -40.0)
    val, ids = torch.topk(t + torch.randn(x.shape, device="cuda", generator=g), k, dim=1)
    drop = torch.rand(ids.shape, device="cuda", generator=g) < 0.2
    odd = torch.arange(k, device="cuda")[None, :] % 2 == 1
    return (torch.where(drop, torch.where(odd, -1, x.shape[1] + 5), ids).to(torch.int32),
            torch.where(drop, torch.where(odd, math.nan, 1e30), val))


def masked(rows, v, kind, fill, seed, part=0.6):
    x = logits(rows, v, kind, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x[torch.rand(x.shape, device="cuda", generator=g) < part] = fill
    x[:, v // 2] = 1.25  # no row of nothing
    return x


def check(x, k, top, tau, what):
    rows, v = x.shape
    tau = torch.tensor(tau).item()  # the interface's fp32: at 1e-7 its rounding is several units of an exponent
    tok = some_tokens(rows, v)
    got = ibwd.token_logprobs_fwd(x, tok, top_n=top, temperature=tau)
    tight_logp_fwd(got, x, tok, top, tau, what)
    g = torch.Generator(device="cuda").manual_seed(3)
    a, h = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)
    lse, ent = got[2], got[1]
    for da, dh in ((a, h), (a, None), (None, h)):
        dx = ibwd.token_logprobs_bwd(x, tok, lse, ent, da, dh, temperature=tau)
        tight_logp_bwd(dx, x, tok, lse, ent, da, dh, tau, what + " bwd")
    ids, teacher = teacher_of(x, k)
    loss, lse = ibwd.distill_fwd(x, ids, teacher, temperature=tau)
    tight_distill(loss, lse, x, ids, teacher, tau, what + " split")
    w = torch.rand(rows, device="cuda", generator=g)
    tight_distill_grad(ibwd.distill_bwd(x, ids, teacher, lse, w, temperature=tau), w, x, ids, teacher, tau,
                       what + " split", lse)
    loss, dx = ibwd.distill_grad(x, ids, teacher, w, temperature=tau)
    tight_distill(loss, None, x, ids, teacher, tau, what + " whole")
    tight_distill_grad(dx, w, x, ids, teacher, tau, what + " whole")


@pytest.mark.parametrize("fill", ["inf", "lowest"])
@pytest.mark.parametrize("rows,v", [(4, 70000), (330, 3001), (700, 1500)])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_masked_logits(rows, v, kind, fill):
    x = masked(rows, v, kind, -INF if fill == "inf" else torch.finfo(DTYPES[kind]).min, seed=rows)
    check(x, 12, 30, 1.0, f"{kind} {fill}")


@pytest.mark.parametrize("k", [7, 513, 1024])
@pytest.mark.parametrize("rows,v", [(2, 40000), (310, 2000)])
def test_padded_slots(rows, v, k):
    for kind in ("bf16", "fp32"):
        check(logits(rows, v, kind, seed=k), k, 3, 1.0, f"K {k}")


@pytest.mark.parametrize("tau", [1e-7, 1e-3, 0.1, 50.0, 1e4])
@pytest.mark.parametrize("kind", ["fp16", "fp32"])
def test_temperatures(tau, kind):
    for rows, v in ((3, 40001), (320, 1500)):
        for fill in (-INF, torch.finfo(DTYPES[kind]).min):
            x = masked(rows, v, kind, fill, seed=14, part=0.4)
            check(x, 12, 9, tau, f"temperature {tau} {fill}")
