"""Plain 64-bit forms of the training operators and the error bounds their
tests hold the kernels to.

Bounds count fp32 roundings of u = 2^-24 each: a sum of n terms loses about
sqrt(n) of them (8 sqrt(n) is taken), an exponential 2^-22 plus what its
argument was rounded by, and the last rounding to the output's type is half a
step of the value."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half the distance of the subnormals: what an underflowing result may be off by."""
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def sum_bound(n):
    return 8 * math.sqrt(n / 32 + 16) * U


def within(got, ref, tol, what):
    """Elementwise |got - ref| <= tol, with NaN and infinities where the reference has them."""
    most = torch.finfo(got.dtype).max * (1 + torch.finfo(got.dtype).eps / 4)
    got, ref = got.double().cpu(), ref.double().cpu()
    ref = torch.where(ref.abs() >= most, ref.sign() * math.inf, ref)  # what the type cannot hold is an infinity
    tol = torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    odd = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[odd], ref[odd]), f"{what}: infinities in other places"
    if not fine.any():
        return
    over = (got[fine] - ref[fine]).abs() - tol[fine]
    assert over.max() <= 0, f"{what}: off by {over.max():.3e} more than the bound {tol[fine][over.argmax()]:.3e}"


# --------------------------------------------------------------- layer norm ---

def norm_fwd(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(-1)
    rstd = ((x - mean[..., None]).square().mean(-1) + eps) ** -0.5
    y = (x - mean[..., None]) * rstd[..., None]
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean, rstd


def check_norm_fwd(got, x, gamma, beta, eps, dtype, what):
    y, mean, rstd = norm_fwd(x, gamma, beta, eps)
    n = x.shape[-1]
    b = sum_bound(n)
    big = x.double().abs().amax(-1)
    g = 1.0 if gamma is None else gamma.double().abs()
    t = 0.0 if beta is None else beta.double().abs()
    # the mean is off by b * big, which moves x - mean; rstd by b and by that shift
    shift = (b + 4 * U) * big
    rel = 2 * b + 8 * U + 2 * shift * rstd
    tol = half_step(dtype) * y.abs() + least(dtype) + ((shift + rel * (x.double() - mean[..., None]).abs().amax(-1)) * rstd)[..., None] * g \
        + 4 * U * t
    within(got[0], y, tol, what + " y")
    if got[1] is not None:
        within(got[1], mean, shift + U * mean.abs(), what + " mean")
        within(got[2], rstd, rel * rstd, what + " rstd")


def norm_bwd(dy, x, mean, rstd, gamma):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double(), rstd.double()
    xh = (x - mean[..., None]) * rstd[..., None]
    d = dy if gamma is None else dy * gamma.double()
    a, b = d.mean(-1, keepdim=True), (d * xh).mean(-1, keepdim=True)
    dx = rstd[..., None] * (d - a - xh * b)
    lead = tuple(range(dy.dim() - 1))
    return dx, (dy * xh).sum(lead), dy.sum(lead), xh, d


def check_norm_bwd(got, dy, x, mean, rstd, gamma, what):
    dx, dgamma, dbeta, xh, d = norm_bwd(dy, x, mean, rstd, gamma)
    n, rows = x.shape[-1], max(1, x.numel() // x.shape[-1])
    r = rstd.double()[..., None]
    if x.numel():
        size = d.abs().mean(-1, keepdim=True) + xh.abs() * (d * xh).abs().mean(-1, keepdim=True)
        tol = half_step(x.dtype) * dx.abs() + least(x.dtype) + r * (sum_bound(n) * size + 8 * U * (d.abs() + size))
        within(got[0], dx, tol, what + " dx")
    if got[1] is not None:
        lead = tuple(range(dy.dim() - 1))
        b = sum_bound(32 * rows) + 8 * U
        within(got[1], dgamma, b * (dy.double() * xh).abs().sum(lead), what + " dgamma")
        within(got[2], dbeta, b * dy.double().abs().sum(lead), what + " dbeta")


# ------------------------------------------------------------------- logits ---

def logp_fwd(x, tokens, top, tau):
    """(logprob, entropy, lse, top_ids, top_logprobs) of [rows, vocab] logits."""
    x = x.double()
    y = x / tau
    lse = torch.logsumexp(y, 1)
    dead = lse == -math.inf
    lp = torch.where(dead[:, None], torch.full_like(y, -math.inf), y - lse[:, None])
    p = lp.exp()
    entropy = -torch.where(p == 0, 0.0, p * lp).sum(1)
    out = [None, entropy, lse]
    if tokens is not None:
        ok = (tokens >= 0) & (tokens < x.shape[1])
        at = torch.where(ok, tokens, 0).long()
        out[0] = torch.where(ok, lp.gather(1, at[:, None])[:, 0], 0.0)
    if top:
        key = torch.where(torch.isnan(x), -math.inf, x)
        ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top]
        free = key.gather(1, ids) == -math.inf
        val = torch.where(free, -math.inf, lp.gather(1, ids))
        val = torch.where(torch.isnan(lse)[:, None] | (lse[:, None] == math.inf), math.nan, val)
        out += [torch.where(free, -1, ids).to(torch.int32), val]
    bad = torch.isnan(lse) | (lse == math.inf)
    for i in range(3):
        if out[i] is not None:
            keep = torch.zeros_like(bad) if i or tokens is None else ~ok
            out[i] = torch.where(bad & ~keep, math.nan, out[i])
    return out


def exp_bound(y, lse, vocab):
    """Relative error of exp(y - lse) computed in fp32 from a row of `vocab` logits."""
    m = torch.where(torch.isfinite(y), y.abs(), 0.0).amax(1) + torch.where(torch.isfinite(lse), lse.abs(), 0.0)
    return sum_bound(vocab) + 64 * U + 4 * U * m


def check_logp_fwd(got, x, tokens, top, tau, what):
    ref = logp_fwd(x, tokens, top, tau)
    y = x.double() / tau
    b = exp_bound(y, ref[2], x.shape[1])
    if tokens is not None:
        within(got[0], ref[0], b + 4 * U * ref[0].abs(), what + " logprob")
    within(got[1], ref[1], b * (2 + ref[1].abs()) * 2, what + " entropy")
    within(got[2], ref[2], b + 4 * U * ref[2].abs(), what + " lse")
    if top:
        assert torch.equal(got[3].cpu(), ref[3].cpu()), what + " top ids"
        within(got[4], ref[4], b[:, None] + 4 * U * ref[4].abs(), what + " top logprobs")


def check_logp_bwd(got, x, tokens, lse, entropy, dlogprob, dentropy, tau, what):
    y, lse = x.double() / tau, lse.double()
    dead = (lse == -math.inf)[:, None]
    lp = torch.where(dead, -math.inf, y - lse[:, None])
    p = lp.exp()
    lpf = torch.where(p == 0, 0.0, lp)
    g = torch.zeros_like(p)
    a = torch.zeros_like(lse)
    if dlogprob is not None:
        ok = (tokens >= 0) & (tokens < x.shape[1])
        a = torch.where(ok & ~dead[:, 0], dlogprob.double(), 0.0)
        g.scatter_add_(1, torch.where(ok, tokens, 0).long()[:, None], a[:, None])
        size = g.abs()
        g -= p * a[:, None]
    else:
        size = g.abs()
    size = size + p * a.abs()[:, None]
    if dentropy is not None:
        h, e = dentropy.double()[:, None], entropy.double()[:, None]
        g -= h * p * (lpf + e)
        size = size + h.abs() * p * (1 + lpf.abs() + e.abs())
    b = exp_bound(y, lse, x.shape[1])[:, None]
    within(got, g / tau, half_step(x.dtype) * (g / tau).abs() + least(x.dtype) + b * size / tau, what)


def targets(ids, teacher, vocab, tau):
    """Probabilities of the kept slots, by slot and by token, and the rows that keep something."""
    ok = (ids >= 0) & (ids < vocab)
    t = torch.where(ok, teacher.double() / tau, -math.inf)
    some = (t > -math.inf).any(1)
    p = torch.where(some[:, None], torch.softmax(t, 1), 0.0)
    full = torch.zeros((ids.shape[0], vocab), dtype=torch.float64, device=ids.device)
    full.scatter_add_(1, torch.where(ok, ids, 0).long(), torch.where(ok, p, 0.0))
    return p, full, some, torch.where(ok, ids, 0).long()


def distill(x, ids, teacher, tau):
    """(loss, lse, d loss / d logits) of [rows, vocab] logits."""
    x = x.double()
    y = x / tau
    lse = torch.logsumexp(y, 1)
    p, full, some, at = targets(ids, teacher, x.shape[1], tau)
    live = some & (lse != -math.inf)
    lq = y - torch.where(lse == -math.inf, 0.0, lse)[:, None]
    gap = torch.where(p > 0, p * (p.log() - lq.gather(1, at)), 0.0)
    loss = torch.where(live, tau * tau * gap.sum(1), 0.0)
    grad = torch.where(live[:, None], tau * (lq.exp() - full), 0.0)
    return loss, lse, grad, p, full, lq


def check_distill(loss, lse, dx, weight, x, ids, teacher, tau, what):
    rl, re, rg, p, full, lq = distill(x, ids, teacher, tau)
    b = exp_bound(x.double() / tau, re, x.shape[1])
    t = torch.where(torch.isfinite(teacher.double()), teacher.double().abs() / tau, 0.0).amax(1)
    b = b + 8 * U * t + sum_bound(ids.shape[1])
    if loss is not None:
        big = torch.where(p > 0, p * (p.log().abs() + torch.where(torch.isfinite(lq), lq.abs(), 0.0).gather(1, torch.where((ids >= 0) & (ids < x.shape[1]), ids, 0).long())), 0.0).sum(1)
        within(loss, rl, tau * tau * (2 * b * (1 + big)), what + " loss")
    if lse is not None:
        within(lse, re, b + 4 * U * re.abs(), what + " lse")
    if dx is not None:
        g = rg * weight.double()[:, None]
        size = tau * weight.double().abs()[:, None] * (lq.exp() + full)
        within(dx, g, half_step(x.dtype) * g.abs() + least(x.dtype) + b[:, None] * size, what + " dlogits")
