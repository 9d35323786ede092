"""Plain 64-bit forms of the norm and rotation of heads, the 8-bit cache and the
attention over it, and the error bounds their tests hold the kernels to.

u = 2^-24 is one fp32 rounding; sums, the last rounding and what an underflow
costs are counted as in train_ref. An angle's cosine and sine: 2 ulp of
sincospif (at most 4 u), the fp32 rounding of at most an eighth of a turn (u), 2^-32
turns of the phase, and 2^-51 of the whole angle for the 53 bits of the frequency and of the
reference's own product. A code times its scale is exact."""
from __future__ import annotations

import math

import torch

from train_ref import U, half_step, least, sum_bound, within

LARGEST = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


# ------------------------------------------------------- norm and rotation ---

def turn(z, angle, start, interleaved, back=False):
    """z [..., H, D] with the pairs from `start` on turned by angle [..., R / 2]."""
    n = angle.shape[-1]
    c, s = angle.cos()[..., None, :], angle.sin()[..., None, :] * (-1 if back else 1)
    y = z.clone()
    i = torch.arange(n, device=z.device)
    a, b = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + i + n)
    y[..., a] = z[..., a] * c - z[..., b] * s
    y[..., b] = z[..., b] * c + z[..., a] * s
    return y


def angles(positions, freq, axes):
    """The pairs' angles of every token, [..., R / 2]; an axis that is none has angle 0."""
    if axes is None:
        return positions.double()[..., None] * freq.double()
    ok = (axes >= 0) & (axes < positions.shape[0])
    p = positions.double()[torch.where(ok, axes, 0).long()].movedim(0, -1)
    return torch.where(ok, p * freq.double(), 0.0)


def pair_sum(v, n, start, interleaved):
    """Of every rotated dimension its own value and its partner's together; others as they are."""
    i = torch.arange(n, device=v.device)
    a, b = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + i + n)
    out = v.clone()
    out[..., a] = out[..., b] = v[..., a] + v[..., b]
    return out


def angle_bound(angle):
    return 5 * U + 2 * math.pi * 2.0 ** -32 + (2.0 ** -51 * angle.abs().amax().item() if angle.numel() else 0.0)


def statistics(x, norm, eps):
    """xh, rstd, and what the kernel's xh may be off by."""
    x = x.double()
    if norm == "none":
        return x, torch.ones_like(x[..., :1]), torch.zeros_like(x)
    b = sum_bound(x.shape[-1])
    shift = torch.zeros_like(x[..., :1])
    if norm == "layer":
        shift = (b + 4 * U) * x.abs().amax(-1, keepdim=True)
        x = x - x.mean(-1, keepdim=True)
    rstd = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    rel = 2 * b + 8 * U + 2 * shift * rstd
    return x * rstd, rstd, shift * rstd + rel * (x * rstd).abs().amax(-1, keepdim=True)


def check_fwd(got, x, norm, gamma, beta, eps, angle, start, interleaved, what):
    xh, _, e = statistics(x, norm, eps)
    g = 1.0 if gamma is None else gamma.double()
    t = 0.0 if beta is None else beta.double()
    z = xh * g + t
    ez = e * abs(g) + 2 * U * (z.abs() + abs(t))
    n = 0 if angle is None else angle.shape[-1]
    y = z if not n else turn(z, angle, start, interleaved)
    if n:
        ez = pair_sum(ez + (angle_bound(angle) + 2 * U) * z.abs(), n, start, interleaved)
    within(got, y, half_step(x.dtype) * y.abs() + least(x.dtype) + ez, what)


def check_bwd(got, dy, x, norm, gamma, eps, angle, start, interleaved, what):
    """got: (dx, dgamma, dbeta)"""
    dy = dy.double()
    n = 0 if angle is None else angle.shape[-1]
    dz, ed = dy, torch.zeros_like(dy)
    if n:
        dz = turn(dy, angle, start, interleaved, back=True)
        ed = pair_sum(torch.zeros_like(dy), n, start, interleaved)
        both = pair_sum(dy.abs(), n, start, interleaved)
        turned = torch.zeros(dy.shape[-1], dtype=torch.bool, device=dy.device)
        turned[start:start + 2 * n] = True
        ed = torch.where(turned, (angle_bound(angle) + 2 * U) * both, 0.0)
    if norm == "none":
        assert got[1] is None and got[2] is None
        within(got[0], dz, half_step(x.dtype) * dz.abs() + least(x.dtype) + ed, what + " dx")
        return
    xh, r, e = statistics(x, norm, eps)
    g = 1.0 if gamma is None else gamma.double()
    d, ed2 = dz * g, ed * abs(g) + U * (dz * g).abs()
    m1 = d.mean(-1, keepdim=True) if norm == "layer" else 0.0
    m2 = (d * xh).mean(-1, keepdim=True)
    dx = r * (d - m1 - xh * m2)
    if x.numel():
        size = (d.abs().mean(-1, keepdim=True) if norm == "layer" else 0.0) + xh.abs() * (d * xh).abs().mean(-1, keepdim=True)
        tol = sum_bound(x.shape[-1]) * size + 8 * U * (d.abs() + size)
        tol = tol + ed2 + (ed2.mean(-1, keepdim=True) if norm == "layer" else 0.0) + xh.abs() * (ed2 * xh.abs()).mean(-1, keepdim=True)
        tol = tol + e * (d * xh).abs().mean(-1, keepdim=True) + xh.abs() * (d.abs() * e).mean(-1, keepdim=True)
        rel = 2 * sum_bound(x.shape[-1]) + 8 * U
        tol = r * tol + (rel + 2 * e) * (r * (d.abs() + size))
        within(got[0], dx, half_step(x.dtype) * dx.abs() + least(x.dtype) + tol, what + " dx")
    lead = tuple(range(x.dim() - 1))
    rows = max(1, x.numel() // x.shape[-1])
    b = sum_bound(32 * rows) + 8 * U
    if got[1] is not None:
        within(got[1], (dz * xh).sum(lead), (b * (dz * xh).abs() + dz.abs() * e + ed * xh.abs()).sum(lead), what + " dgamma")
    if got[2] is not None:
        assert norm == "layer"
        within(got[2], dz.sum(lead), (b * dz.abs() + ed).sum(lead), what + " dbeta")


# -------------------------------------------------------------------- cache ---

def scale_for(amax, code):
    """The least power of two at which amax is no larger than the largest code, for one number."""
    if amax == 0:
        return 2.0 ** -126
    e = -126
    m, e = math.frexp(amax / LARGEST[code])
    e = e - 1 if m == 0.5 else e
    while LARGEST[code] * 2.0 ** e < amax:
        e += 1
    while e > -126 and LARGEST[code] * 2.0 ** (e - 1) >= amax:
        e -= 1
    return 2.0 ** max(-126, min(120, e))


def encode(v, code):
    """Codes (as numbers) of float64 values in units of the scale."""
    v = v.clamp(-LARGEST[code], LARGEST[code])
    if code == torch.int8:
        return torch.round(torch.nan_to_num(v, nan=0.0))
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    step = torch.where(v.abs() >= 16 * step, 2 * step, step)  # (should log2 have rounded down)
    return torch.round(v / step) * step


def positions_of(lens, cu, table, page):
    """(sequence, packed token, position) of every packed token that has a place."""
    width = table.shape[1] * page
    out = []
    for b, n in enumerate(lens):
        first, last = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
        for i in range(first, last):
            at = n - (last - i)
            if 0 <= at < width:
                out.append((b, i, at))
    return out


def write_ref(x, codes, scale, table, lens, cu, page):
    """Codes (float64) and scales of a cache (CPU tensors) after x [N, H, D] was written."""
    codes_t = codes.dtype
    held, unit = codes.double(), scale.double().clone()
    blocks = {}
    for b, i, at in positions_of(lens, cu, table, page):
        p = int(table[b, at // page])
        if 0 <= p < codes.shape[0]:
            blocks.setdefault(p, []).append((at % page, i))
    for p, tokens in blocks.items():
        slots = [s for s, _ in tokens]
        for h in range(x.shape[1]):
            v = torch.stack([x[i, h] for _, i in tokens]).double()
            fine = v[torch.isfinite(v)].abs()
            u = scale_for(fine.max().item() if fine.numel() else 0.0, codes_t)
            lo = min(slots)
            old = unit[p, h].item()
            if lo:
                u = max(u, old) if old == old else u
                held[p, h, :lo] = encode(held[p, h, :lo] * (old / u), codes_t)
            for s, row in zip(slots, v):
                held[p, h, s] = encode(row / u, codes_t)
            bad = codes_t == torch.int8 and (bool(torch.isnan(v).any()) or (lo and old != old))
            unit[p, h] = math.nan if bad else u
    return held, unit


def read_ref(codes, scale, table, lens, length, page):
    out = torch.zeros((len(lens), length, codes.shape[1], codes.shape[3]), dtype=torch.float64, device=codes.device)
    held = codes.float().double() * scale.double()[:, :, None, None]
    for b, n in enumerate(lens):
        for at in range(0, min(max(n, 0), length, table.shape[1] * page), page):
            p, end = int(table[b, at // page]), min(at + page, n, length)
            if 0 <= p < codes.shape[0]:
                out[b, at:end] = held[p, :, :end - at].transpose(0, 1)
    return out


def check_attention(got, q, k_codes, v_codes, k_scale, v_scale, table, lens, cu, select, scale, page, what):
    """Every packed token that belongs to a sequence; got: (out, lse)."""
    n_heads, d = k_codes.shape[1], k_codes.shape[3]
    group = q.shape[1] // n_heads
    width = table.shape[1] * page
    code = LARGEST[v_codes.dtype]
    for b, n in enumerate(lens):
        first, last = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
        held = min(max(n, 0), width)
        ids = torch.arange(held, device=q.device)
        pages = table[b].long()[ids // page]
        good = (pages >= 0) & (pages < k_codes.shape[0])
        pages = torch.where(good, pages, 0)
        k, v = (c[pages, :, ids % page].float().double() * s[pages].double()[..., None] for c, s in ((k_codes, k_scale), (v_codes, v_scale)))
        vs = v_scale[pages].double()
        for i in range(first, last):
            seen = min(max(0, n - (last - 1 - i)), held)
            if select is None:
                at = ids[:seen][good[:seen]]
            else:
                at = select[i].long()
                at = at[(at >= 0) & (at < seen)]
                at = at[good[at]]
            x = q[i].double().view(n_heads, group, d)
            kk, vv = k[at].transpose(0, 1), v[at].transpose(0, 1)          # [H, L, D]
            name = f"{what} token {i}"
            if not len(at):
                within(got[0][i], torch.zeros_like(q[i]), 0.0, name)
                assert (got[1][i] == -math.inf).all(), name
                continue
            y = x @ kk.transpose(1, 2) * scale                              # [H, G, L]
            lse = torch.logsumexp(y, -1)
            p = torch.softmax(y, -1)
            out = p @ vv
            # logits: the query in fp16 of its largest entry (2^-25 of it at least, 2^-11 of an entry of 11 bits none), sums of D
            # products by tensor cores, each step of 16 off by an ulp, and a few roundings
            ds = abs(scale) * (2.0 ** -24 * x.abs().amax(-1)[..., None] * kk.abs().sum(-1)[:, None]
                          + (d / 8 + 8) * 2 * U * (x.abs() @ kk.abs().transpose(1, 2))) + 8 * U * (y.abs() + 1)
            dm = ds.amax(-1)
            m = y.amax(-1)
            ln = sum_bound(len(at)) + 2.0 ** -20
            within(got[1][i].view(n_heads, group), lse, dm + ln + 4 * U * (lse.abs() + m.abs()), name + " lse")
            # weights: fp16, 2^-11; those below 2^-29 of the largest lose bits and vanish
            rel = 2 * dm + 2.0 ** -11 + 2.0 ** -20 + (len(at) / 16 + 64) * 2 * U
            tiny = 2.0 ** -39 * (p * vs[at].T[:, None]).amax(-1) * code * len(at)
            tol = half_step(q.dtype) * out.abs() + least(q.dtype) + rel[..., None] * (p @ vv.abs()) + tiny[..., None]
            within(got[0][i].view(n_heads, group, d), out, tol, name)
