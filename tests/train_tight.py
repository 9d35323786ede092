"""Bounds of the operators over logits that stay small on rows with masked
logits and padded slots: what a value may be off by counts only what reaches it.

u = 2^-24 is one fp32 rounding.  With m the row's largest logit, a kernel's
exponent is (x - m) log2(e) / T: a handful of roundings of that difference, not
of x, so that a masked logit costs nothing but its own log probability a
relative error.  sum_bound(n) is what a sum of n terms may lose, 64 u more what
its exponentials do (2^-22 each, and their arguments' roundings weighed by the
exponentials themselves, whose mean argument is at most log n).
"""
from __future__ import annotations

import math

import torch

from train_ref import U, distill, half_step, least, logp_fwd, sum_bound, targets, within

TINY = 1e-37  # exponentials below fp32's normal range are flushed to 0


def _row(x, tau):
    """Largest logit / T (0 where there is none), and what the row's sum of exponentials is off by, relatively."""
    m = x.double().amax(1)
    m = torch.where(torch.isfinite(m), m, 0.0) / tau
    return m, sum_bound(x.shape[1]) + 64 * U + 8 * U * math.log(x.shape[1] + 1)


def _lse_tol(x, lse, tau):
    m, b = _row(x, tau)
    return b + 4 * U * (m.abs() + torch.where(torch.isfinite(lse), lse.abs(), 0.0))


def _lp_tol(x, lp):
    b = sum_bound(x.shape[1]) + 64 * U + 8 * U * math.log(x.shape[1] + 1)
    return b + 8 * U * (1 + lp.abs())


def tight_logp_fwd(got, x, tokens, top, tau, what):
    ref = logp_fwd(x, tokens, top, tau)
    if tokens is not None:
        within(got[0], ref[0], _lp_tol(x, ref[0]), what + " logprob")
    _, b = _row(x, tau)
    within(got[1], ref[1], 4 * b * (1 + ref[1].abs() + math.log(x.shape[1] + 1)), what + " entropy")
    within(got[2], ref[2], _lse_tol(x, ref[2], tau), what + " lse")
    if top:
        assert torch.equal(got[3].cpu(), ref[3].cpu()), what + " top ids"
        within(got[4], ref[4], _lp_tol(x, ref[4]), what + " top logprobs")


def _q(x, lse, tau):
    """log q and q for a given lse, and the relative error of q: roundings of the exponent (of which only those
    above fp32's smallest exponentials count) and of lse T."""
    lse = lse.double()
    dead = (lse == -math.inf)[:, None]
    lq = torch.where(dead, -math.inf, x.double() / tau - torch.where(dead[:, 0], 0.0, lse)[:, None])
    b = 64 * U + 8 * U * torch.clamp(lq.abs(), max=200.0)
    return lq, lq.exp(), b


def tight_logp_bwd(got, x, tokens, lse, entropy, dlogprob, dentropy, tau, what):
    lq, q, b = _q(x, lse, tau)
    lqf = torch.where(q == 0, 0.0, lq)
    dead = lse == -math.inf
    g = torch.zeros_like(q)
    a = torch.zeros_like(lse, dtype=torch.float64)
    if dlogprob is not None:
        ok = (tokens >= 0) & (tokens < x.shape[1])
        a = torch.where(ok & ~dead, dlogprob.double(), 0.0)
        g.scatter_add_(1, torch.where(ok, tokens, 0).long()[:, None], a[:, None])
    size = g.abs() + q * a.abs()[:, None]
    g -= q * a[:, None]
    coef = a.abs()[:, None]
    if dentropy is not None:
        h, e = torch.where(dead, 0.0, dentropy.double())[:, None], entropy.double()[:, None]
        g -= h * q * (lqf + e)
        size = size + h.abs() * q * (1 + lqf.abs() + e.abs())
        coef = coef + 200 * h.abs()
    g = g / tau
    within(got, g, half_step(x.dtype) * g.abs() + least(x.dtype) + (b * size + TINY * coef) / tau, what)


def tight_distill(loss, lse, x, ids, teacher, tau, what):
    rl, re, _, p, _, _ = distill(x, ids, teacher, tau)
    v = x.shape[1]
    ok = (ids >= 0) & (ids < v) & (p > 0)
    m, b = _row(x, tau)
    t = torch.where(ok, teacher.double(), -math.inf)
    tm = t.amax(1, keepdim=True)
    dt = torch.where(ok, t - torch.where(torch.isfinite(tm), tm, 0.0), 0.0) / tau
    xk = x.double().gather(1, torch.where(ok, ids, 0).long()) / tau - m[:, None]
    dx = torch.where(ok & torch.isfinite(xk), xk, 0.0)
    k = sum_bound(ids.shape[1]) + 64 * U
    # of the sum over the slots, of the probabilities (off by 4 u |dt| + k), and of the two logarithms
    tol = (k + 4 * U * torch.where(ok, dt.abs(), 0.0).amax(1)) * (1 + (p * (dt.abs() + dx.abs())).sum(1))
    tol = tol + b + 8 * U * (math.log(v + 1) + math.log(ids.shape[1] + 1))
    if loss is not None:
        within(loss, rl, tau * tau * tol, what + " loss")
    if lse is not None:
        within(lse, re, _lse_tol(x, re, tau), what + " lse")


def tight_distill_grad(dx, weight, x, ids, teacher, tau, what, lse=None):
    """lse: as a separate backward pass was given it, else the row's own."""
    v = x.shape[1]
    p, full, some, _ = targets(ids, teacher, v, tau)
    own = lse is None
    if own:
        lse = torch.logsumexp(x.double() / tau, 1)
    live = (some & (lse != -math.inf))[:, None]
    lq, q, b = _q(x, lse, tau)
    if own:
        b = b + _row(x, tau)[1]
    w = weight.double()[:, None]
    g = torch.where(live, tau * w * (q - full), 0.0)
    k = sum_bound(ids.shape[1]) + 64 * U + 4 * U * 100  # (a teacher's exponent is over -100 where p counts)
    tol = half_step(x.dtype) * g.abs() + least(x.dtype) + tau * w.abs() * (b * q + k * full + TINY)
    within(dx, g, tol, what + " dlogits")
