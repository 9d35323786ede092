"""Cases of the operators between the projections of queries, keys and values
and what reads them: the norm of each head with the position rotation in the
same pass, forward and backward; a paged cache of 8-bit keys and values,
written and read back; and the attention over such a cache, over all of a
sequence's tokens or over those that an indexer selected.

Each case is one call as a training loop or a server makes it (a write is
followed by reading the sequences back); `run` computes it in elementary torch
operations, or through this package where `own` is set.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LARGEST = {"e4m3": 448.0, "int8": 127.0}
EPS = 1e-6


def _rope(op, **kw):
    base = dict(op=op, tokens=1, heads=1, kv_heads=0, dim=128, rotated=128, start=0, axes=1, interleaved=False, q_norm="rms",
                k_norm="rms", type="bf16", dy="bf16", far=4096, fused=True)
    return {**base, **kw}


def _cache(op, **kw):
    base = dict(op=op, batch=1, shortest=1, longest=64, kv_heads=8, dim=128, page=64, code="e4m3", type="bf16", empty=False)
    return {**base, **kw}


def listed():
    return [
        # one decoding step of 8 sequences far into their contexts: latency alone
        _rope("rope", name="rope_step", tokens=8, heads=32, kv_heads=8, far=200000),
        # a clip's patches with time, height and width, an odd number of them, adjacent pairs
        _rope("rope", name="rope_video", tokens=16381, heads=24, kv_heads=8, axes=3, interleaved=True, type="fp16", far=512),
        # a training batch's attention heads back to the fused projection
        _rope("rope_bwd", name="rope_heads_bwd", tokens=8192, heads=32, kv_heads=8, far=8192),
        # the anchor's indexer: dQ and dK (fp32) back through a partial rotation and the keys' layer norm
        _rope("rope_bwd", name="rope_index_bwd", tokens=4096, heads=64, kv_heads=1, rotated=64, q_norm="none", k_norm="layer",
              dy="fp32", far=4096, fused=False),
        # one decoding step of an indexer: a key for each of 16 sequences is written, all are read back for its scores
        _cache("write", name="write_step", batch=16, shortest=700, longest=4096, kv_heads=1, new=1, values=False),
        # prompts of all lengths are written, keys and values, and read back
        _cache("write", name="write_prompts", batch=16, shortest=33, longest=2048, kv_heads=8, new=0, values=True),
        # an indexer's keys of long contexts
        _cache("read", name="read_index", batch=4, shortest=9001, longest=32768, kv_heads=1),
        # values in whole numbers, heads of an odd number, ragged
        _cache("read", name="read_int8", batch=7, shortest=100, longest=16384, kv_heads=5, code="int8", page=32, type="fp16"),
        # one decoding step of short contexts: latency
        _cache("attend", name="attend_step", batch=8, shortest=100, longest=1000, group=4, new=1, select=0),
        # one decoding step of a large ragged batch
        _cache("attend", name="attend_batch", batch=64, shortest=37, longest=16384, group=4, new=1, select=0),
        # four drafted tokens and the one before them, behind long contexts
        _cache("attend", name="attend_draft", batch=2, shortest=60000, longest=131072, kv_heads=4, group=6, new=5, select=0,
               code="int8", page=16),
        # what an indexer selected for each of 64 tokens: 2048 of up to 65536 positions, one head of keys
        _cache("attend", name="attend_select", batch=64, shortest=1500, longest=65536, kv_heads=1, group=16, new=1, select=2048),
    ]


def _size(rng, lo, hi, multiple=1):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, n // multiple * multiple)


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "write", "read", "attend", "attend"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("rope", "rope_bwd"):
        dim = rng.choice([64, 128, 128, 256, _size(rng, 16, 256, rng.choice([1, 2, 8]))])
        heads, kv = rng.choice([1, 4, 12, 32, 64]), rng.choice([0, 1, 2, 5, 8])
        axes = rng.choice([1, 1, 2, 3])
        rotated = rng.choice([dim // 2 * 2, dim // 4 * 2])
        return _rope(op, tokens=_size(rng, 1, min(16384, (1 << 26) // (dim * (heads + kv)))), heads=heads, kv_heads=kv, dim=dim,
                     rotated=rotated, start=rng.choice([0, dim - rotated]), axes=axes, interleaved=rng.random() < 0.4,
                     q_norm=rng.choice(["rms", "rms", "layer", "none"]), k_norm=rng.choice(["rms", "layer"]), type=kind,
                     dy=rng.choice([kind, "fp32"]), far=_size(rng, 1000, 500000), fused=rng.random() < 0.6)
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 5, 8])
    batch = _size(rng, 1, 64)
    common = dict(batch=batch, kv_heads=kv, page=page, code=rng.choice(["e4m3", "e4m3", "int8"]), empty=rng.random() < 0.2)
    if op == "attend":
        dim = rng.choice([64, 128, 128, 256])
        kind = rng.choice(["bf16", "bf16", "fp16"])
        group, new = rng.choice([1, 3, 4, 8, 16]), rng.choice([1, 1, 1, 2, 4, 7])
        longest = _size(rng, 16, min(65536, (1 << 29) // max(1, group * new // 8) // (batch * kv * dim)))
        select = rng.choice([0, 0, _size(rng, 1, min(2048, 2 * longest))])
        if select:
            select = max(1, min(select, (1 << 27) // (batch * new * kv * dim)))
        return _cache(op, longest=longest, shortest=rng.choice([1, max(1, longest // 2)]), dim=dim, type=kind,
                      group=group, new=new, select=select, **common)
    dim = rng.choice([32, 64, 80, 128, 256])
    longest = _size(rng, 1, min(16384, (1 << 24) // (batch * kv * dim)))
    case = _cache(op, longest=longest, shortest=rng.choice([1, max(1, longest // 2)]), dim=dim, type=kind, **common)
    if op == "write":
        case.update(new=rng.choice([0, 1, 3, 100]), values=rng.random() < 0.7)
    return case


# ------------------------------------------------------------------ inputs ---

def _heads(g, tokens, heads, dim, kind, width=None, at=0):
    """[tokens, heads, dim] of heads of different size, as columns of a wider projection where `width` is given."""
    x = torch.empty((tokens, heads, dim), device="cuda").normal_(generator=g)
    x.mul_(torch.rand((1, heads, 1), device="cuda", generator=g) * 2 + 0.25)
    if kind is None:
        return x
    if width is None:
        return x.to(TYPES[kind])
    buf = torch.empty((tokens, width), device="cuda", dtype=TYPES[kind])
    out = buf[:, at:at + heads * dim].view(tokens, heads, dim)
    out.copy_(x)
    return out


def _prepare_rope(case, g, s):
    t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    width = (hq + 2 * hk) * d if case["fused"] else None
    for name, heads, at in (("q", hq, 0), ("k", hk, hq * d)):
        norm = case[name + "_norm"]
        s[name] = _heads(g, t, heads, d, case["type"], width, at) if heads else None
        weights = heads and norm != "none"
        s[name + "_gamma"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=g) if weights else None
        s[name + "_beta"] = 0.2 * torch.randn(d, device="cuda", generator=g) if weights and norm == "layer" else None
        if case["op"] == "rope_bwd":
            s["d" + name] = _heads(g, t, heads, d, case["dy"]) if heads else None
    n = case["rotated"] // 2
    s["inv_freq"] = 10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / max(1, n))
    if case["axes"] == 1:
        # sequences packed behind one another, each from a place of its own
        first = torch.randint(0, case["far"], (8,), device="cuda", generator=g)
        at = torch.arange(t, device="cuda")
        s["positions"] = (first[at * 8 // max(1, t)] + at % max(1, -(-t // 8))).to(torch.int32)
        s["axes"] = None
    else:
        s["positions"] = torch.randint(0, case["far"], (case["axes"], t), device="cuda", generator=g, dtype=torch.int32)
        s["axes"] = (torch.arange(n, device="cuda") * case["axes"] // max(1, n)).to(torch.int32)


def _scale_of(amax, code):
    """The least power of two at which nothing up to amax is beyond the codes."""
    most, power = math.frexp(LARGEST[code])
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1
    e = e - power + (m > most)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(-126, 120)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _code(x, code):
    """x in units of the scale, to the nearest code, ties to even."""
    x = x.clamp(-LARGEST[code], LARGEST[code])
    return torch.round(x).to(torch.int8) if code == "int8" else x.to(CODES[code])


def _fill(g, pages, heads, page, dim, code, loud):
    """A cache's pages with keys or values in them: some channels are louder than others."""
    cache = torch.empty((pages, heads, page, dim), device="cuda", dtype=CODES[code])
    scale = torch.empty((pages, heads), device="cuda")
    step = max(1, (1 << 25) // (heads * page * dim))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.empty((n, heads, page, dim), device="cuda").normal_(generator=g)
        x *= loud
        scale[a:a + n] = _scale_of(x.abs().amax((2, 3)), code)
        cache[a:a + n] = _code(x / scale[a:a + n, :, None, None], code)
    return cache, scale


def _lengths(case):
    """Each sequence's tokens, spread evenly over their logarithm, and how many of them the call brings."""
    b, lo, hi = case["batch"], case["shortest"], case["longest"]
    lens = [round(lo * (hi / lo) ** (1 - i / max(1, b - 1))) for i in range(b)]
    if case["empty"] and b > 1:  # a place of a padded batch without a sequence
        lens[-1] = 0
    if case.get("new", 1) == 1:  # no offsets: one token for each place
        return lens, [1] * b
    if case["new"] == 0:
        return lens, list(lens)
    return lens, [min(n, case["new"] - i % case["new"]) for i, n in enumerate(lens)]  # some bring fewer


def _prepare_cache(case, g, s):
    b, h, d, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    order = torch.randperm(b, device="cuda", generator=g)
    lens, new = (torch.tensor(x, device="cuda")[order] for x in _lengths(case))
    count = (lens + page - 1) // page
    total, width = int(count.sum()), -(-case["longest"] // page)
    order = torch.randperm(total + 3, device="cuda", generator=g)
    at = torch.arange(width, device="cuda")[None]
    row = (torch.cumsum(count, 0) - count)[:, None] + at
    table = torch.where(at < count[:, None], order[torch.where(at < count[:, None], row, torch.zeros_like(row))], -1)
    s["table"], s["lens"] = table.to(torch.int32).contiguous(), lens.to(torch.int32)
    loud = torch.exp(0.5 * torch.randn(d, device="cuda", generator=g))
    values = case["op"] == "attend" or (case["op"] == "write" and case["values"])
    s["k_cache"], s["k_scale"] = _fill(g, total + 3, h, page, d, case["code"], loud)
    s["v_cache"], s["v_scale"] = _fill(g, total + 3, h, page, d, case["code"], 1.0) if values else (None, None)
    if case["op"] == "read":
        return
    s["cu"] = None
    n = b
    if case["new"] != 1:
        s["cu"] = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)]).to(torch.int32)
        n = int(s["cu"][-1])
    if case["op"] == "write":
        s["k"] = (_heads(g, n, h, d, None) * loud).to(TYPES[case["type"]])
        s["v"] = _heads(g, n, h, d, case["type"]) if values else None
        return
    group = case["group"]
    s["q"] = (1.5 * _heads(g, n, h * group, d, None) / loud).to(TYPES[case["type"]])
    s["select"] = None
    if case["select"]:
        # distinct positions of each token's own context, in no order; -1 where it has fewer
        seq, seen = _visible(s, n)
        k = case["select"]
        start = torch.randint(0, 1 << 30, (n, 1), device="cuda", generator=g)
        stride = torch.clamp(seen // k, min=1)[:, None]
        i = torch.arange(k, device="cuda")[None]
        ids = (start + i * stride) % torch.clamp(seen, min=1)[:, None]
        ids = torch.where(i < seen[:, None], ids, -1)
        s["select"] = ids[:, torch.randperm(k, device="cuda", generator=g)].to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case)
    (_prepare_rope if case["op"] in ("rope", "rope_bwd") else _prepare_cache)(case, g, s)
    return s


# ------------------------------------------------------------- plain forms ---

def _turn(z, cos, sin, start, interleaved):
    """Rotates pairs of z [T, H, D] by the angles of cos and sin [T, 1, R / 2]."""
    r = 2 * cos.shape[-1]
    y = z.clone()
    part = z[..., start:start + r]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        y[..., start:start + r:2] = a * cos - b * sin
        y[..., start + 1:start + r:2] = b * cos + a * sin
    else:
        a, b = part[..., :r // 2], part[..., r // 2:]
        y[..., start:start + r // 2] = a * cos - b * sin
        y[..., start + r // 2:start + r] = b * cos + a * sin
    return y


def _angles(s):
    p = s["positions"].double()
    angle = (p[:, None] if s["axes"] is None else p[s["axes"].long()].T) * s["inv_freq"]
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _normed(x, norm):
    x = x.float()
    if norm == "none":
        return x, None
    n = x.shape[-1]
    if norm == "layer":
        x = x - x.sum(-1, keepdim=True) / n
    rstd = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + EPS)
    return x * rstd, rstd


def _rope_fwd(x, gamma, beta, norm, cos, sin, case):
    z, _ = _normed(x, norm)
    if gamma is not None:
        z = z * gamma
    if beta is not None:
        z = z + beta
    return _turn(z, cos, sin, case["start"], case["interleaved"]).to(x.dtype)


def _rope_bwd(dy, x, gamma, norm, cos, sin, case):
    dz = _turn(dy.float(), cos, -sin, case["start"], case["interleaved"])
    if norm == "none":
        return dz.to(x.dtype), None, None
    xh, rstd = _normed(x, norm)
    n = x.shape[-1]
    d = dz * gamma
    dx = d - xh * ((d * xh).sum(-1, keepdim=True) / n)
    if norm == "layer":
        dx = dx - d.sum(-1, keepdim=True) / n
    dx = (dx * rstd).to(x.dtype)
    return dx, (dz * xh).sum((0, 1)), dz.sum((0, 1)) if norm == "layer" else None


def _plain_rope(s):
    c = s["case"]
    cos, sin = _angles(s)
    if c["op"] == "rope":
        yq = _rope_fwd(s["q"], s["q_gamma"], s["q_beta"], c["q_norm"], cos, sin, c)
        yk = None if s["k"] is None else _rope_fwd(s["k"], s["k_gamma"], s["k_beta"], c["k_norm"], cos, sin, c)
        return {"q": yq, "k": yk}
    dq, gq, bq = _rope_bwd(s["dq"], s["q"], s["q_gamma"], c["q_norm"], cos, sin, c)
    dk, gk, bk = (None, None, None) if s["k"] is None else _rope_bwd(s["dk"], s["k"], s["k_gamma"], c["k_norm"], cos, sin, c)
    return {"q": dq, "k": dk, "q_gamma": gq, "q_beta": bq, "k_gamma": gk, "k_beta": bk}


def _tokens(s, n):
    """Of each packed token its sequence and its position there."""
    if s["cu"] is None:
        return torch.arange(n, device="cuda"), s["lens"].long() - 1
    cu = s["cu"].long()
    at = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu, at, right=True) - 1
    return seq, s["lens"].long()[seq] - (cu[seq + 1] - at)


def _visible(s, n):
    seq, at = _tokens(s, n)
    return seq, at + 1


def _write(x, cache, scale, s, code):
    """Writes x [N, H, D] into the cache's pages; a page keeps its scale, or gets a larger one and its older tokens with it."""
    page = cache.shape[2]
    seq, at = _tokens(s, x.shape[0])
    on = at >= 0
    seq, at, x = seq[on], at[on], x[on].float()
    where = s["table"].long()[seq, at // page]
    slot = at % page
    amax = torch.zeros_like(scale).scatter_reduce_(0, where[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    first = torch.full((scale.shape[0],), page, device="cuda").scatter_reduce_(0, where, slot, "amin")
    need = _scale_of(amax, code)
    old = first < page  # pages of this call
    kept = torch.where((first > 0)[:, None], torch.maximum(scale, need), need)
    factor = scale / kept
    pages = torch.nonzero(old & (first > 0) & (factor < 1).any(1))[:, 0]
    older = cache[pages].float() * factor[pages][:, :, None, None]
    older = torch.where((torch.arange(page, device="cuda") < first[pages][:, None])[:, None, :, None], older, cache[pages].float())
    cache[pages] = _code(older, code)
    scale.copy_(torch.where(old[:, None], kept, scale))
    bits = cache.view(torch.uint8)
    bits[where, :, slot] = _code(x / scale[where][:, :, None], code).view(torch.uint8)


def _read(cache, scale, s, length, dtype):
    page = cache.shape[2]
    at = torch.arange(length, device="cuda")
    ok = at[None] < s["lens"][:, None]
    where = torch.where(ok, s["table"].long()[:, at // page], 0)
    x = cache.view(torch.uint8)[where, :, at % page].view(cache.dtype).float() * scale[where][..., None]
    return torch.where(ok[..., None, None], x, torch.zeros((), device="cuda")).to(dtype)


def _attend(q, k, v, ok, scale):
    """q [N, H, G, D], k and v [N, L, H, D], ok [N, ..., L] -> [N, H, G, D] and log-sum-exp."""
    y = torch.einsum("nhgd,nlhd->nhgl", q, k) * scale
    y = torch.where(ok, y, torch.full((), -math.inf, device="cuda"))
    m = y.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(y - m)
    z = e.sum(-1, keepdim=True)
    some = z > 0
    p = e / torch.where(some, z, torch.ones_like(z))
    return torch.einsum("nhgl,nlhd->nhgd", p, v), (m + torch.log(z))[..., 0]


def _plain_attend(s):
    c = s["case"]
    q, h, d = s["q"], c["kv_heads"], c["dim"]
    n, hq = q.shape[0], q.shape[1]
    group, page = hq // h, c["page"]
    seq, seen = _visible(s, n)
    q32 = q.float().view(n, h, group, d)
    if s["select"] is not None:
        ids = s["select"].long()
        ok = (ids >= 0) & (ids < seen[:, None])
        ids = torch.where(ok, ids, torch.zeros_like(ids))
        where = torch.where(ok, s["table"].long()[seq[:, None], ids // page], 0)
        k, v = (x.view(torch.uint8)[where, :, ids % page].view(x.dtype).float() * y[where][..., None]
                for x, y in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
        o, lse = _attend(q32, k, v, ok[:, None, None], d ** -0.5)
        return o.reshape(n, hq, d).to(q.dtype), lse.reshape(n, hq)
    k = _read(s["k_cache"], s["k_scale"], s, c["longest"], torch.float32)
    v = _read(s["v_cache"], s["v_scale"], s, c["longest"], torch.float32)
    at = torch.arange(c["longest"], device="cuda")
    if s["cu"] is None:
        o, lse = _attend(q32, k, v, (at < seen[:, None])[:, None, None], d ** -0.5)
        return o.reshape(n, hq, d).to(q.dtype), lse.reshape(n, hq)
    # the sequences' tokens side by side, as many places as the longest has
    most = c["new"]
    place = torch.arange(n, device="cuda") - s["cu"].long()[seq]
    wide = torch.zeros((c["batch"], most, h, group, d), device="cuda")
    wide[seq, place] = q32
    limit = torch.zeros((c["batch"], most), device="cuda", dtype=torch.long)
    limit[seq, place] = seen
    ok = (at < limit[..., None])[:, None, :, None].expand(-1, h, -1, group, -1).reshape(c["batch"], h, most * group, -1)
    o, lse = _attend(wide.transpose(1, 2).reshape(c["batch"], h, most * group, d), k, v, ok, d ** -0.5)
    o = o.view(c["batch"], h, most, group, d).transpose(1, 2)[seq, place]
    lse = lse.view(c["batch"], h, most, group).transpose(1, 2)[seq, place]
    return o.reshape(n, hq, d).to(q.dtype), lse.reshape(n, hq)


def _plain(s):
    c = s["case"]
    if c["op"] in ("rope", "rope_bwd"):
        return _plain_rope(s)
    if c["op"] == "attend":
        return _plain_attend(s)
    dt = TYPES[c["type"]]
    if c["op"] == "read":
        return _read(s["k_cache"], s["k_scale"], s, c["longest"], dt)
    _write(s["k"], s["k_cache"], s["k_scale"], s, c["code"])
    out = [_read(s["k_cache"], s["k_scale"], s, c["longest"], dt), s["k_scale"]]
    if s["v"] is not None:
        _write(s["v"], s["v_cache"], s["v_scale"], s, c["code"])
        out += [_read(s["v_cache"], s["v_scale"], s, c["longest"], dt), s["v_scale"]]
    return out


# ------------------------------------------------------ the framework's calls ---

def _own(s):
    import sparse_attention_indexer_bwd_gb300 as ibwd
    c = s["case"]
    if c["op"] in ("rope", "rope_bwd"):
        how = dict(q_norm=c["q_norm"], k_norm=c["k_norm"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS, axes=s["axes"],
                   start=c["start"], interleaved=c["interleaved"])
        if c["op"] == "rope":
            yq, yk = ibwd.qk_norm_rope_fwd(s["q"], s["k"], s["positions"], s["inv_freq"], q_beta=s["q_beta"], k_beta=s["k_beta"],
                                           **how)
            return {"q": yq, "k": yk}
        out = ibwd.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["inv_freq"], **how)
        return dict(zip(("q", "k", "q_gamma", "q_beta", "k_gamma", "k_beta"), out))
    table, lens = s["table"], s["lens"]
    if c["op"] == "attend":
        return ibwd.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], table, lens, cu=s["cu"],
                                    select=s["select"])
    dt = TYPES[c["type"]]
    if c["op"] == "read":
        return ibwd.cache_read(s["k_cache"], s["k_scale"], table, lens, c["longest"], dtype=dt)
    ibwd.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], table, lens, cu=s["cu"])
    out = [ibwd.cache_read(s["k_cache"], s["k_scale"], table, lens, c["longest"], dtype=dt), s["k_scale"]]
    if s["v"] is not None:
        out += [ibwd.cache_read(s["v_cache"], s["v_scale"], table, lens, c["longest"], dtype=dt), s["v_scale"]]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------- work and 64-bit results ---

def work(case):
    size = {"fp32": 4, "bf16": 2, "fp16": 2}
    e, d, kv = size[case["type"]], case["dim"], case["kv_heads"]
    if case["op"] in ("rope", "rope_bwd"):
        n = case["tokens"] * (case["heads"] + kv) * d
        per = 2 * e if case["op"] == "rope" else 2 * e + size[case["dy"]]
        return {"bytes": n * per + 4 * case["tokens"] * case["axes"], "flops": (12 if case["op"] == "rope" else 20) * n}
    lens, new = _lengths(case)
    tokens, padded = sum(lens), case["batch"] * case["longest"]
    if case["op"] == "read":
        return {"bytes": tokens * kv * d + padded * kv * d * e, "flops": tokens * kv * d}
    if case["op"] == "write":
        both = 2 if case["values"] else 1
        brought = sum(min(n, m) for n, m in zip(lens, new))
        return {"bytes": both * kv * d * (brought * (e + 1) + tokens + padded * e), "flops": both * kv * d * (3 * brought + tokens)}
    rows, group, most = sum(new), case["group"], case["select"]
    read = sum(m * min(n, most) for n, m in zip(lens, new)) if most else tokens
    pairs = read if most else sum(m * n for n, m in zip(lens, new))
    return {"bytes": read * kv * 2 * d + rows * kv * group * d * 2 * e, "flops": 4 * pairs * kv * group * d}


def _rotation(case, s):
    """The rotation of every token as complex factors, with the dimensions that each turns."""
    n = case["rotated"] // 2
    if n == 0:
        return None
    a = torch.arange(n, device="cuda")
    first = case["start"] + (2 * a if case["interleaved"] else a)
    second = first + (1 if case["interleaved"] else n)
    pos = s["positions"].double().reshape(case["axes"], -1)
    pick = torch.zeros(n, dtype=torch.long, device="cuda") if s["axes"] is None else s["axes"].long()
    return torch.exp(1j * (s["inv_freq"][:, None] * pos[pick]).T)[:, None], first, second


def _rotated(z, rot, back=False):
    if rot is None:
        return z
    w, i, j = rot
    pair = torch.complex(z[..., i], z[..., j]) * (w.conj() if back else w)
    out = z.clone()
    out[..., i], out[..., j] = pair.real, pair.imag
    return out


def _exact_rope(case, s):
    rot = _rotation(case, s)
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            out[name] = None
            continue
        norm, gamma, beta = case[name + "_norm"], s[name + "_gamma"], s[name + "_beta"]
        x = s[name].double()
        mean = x.mean(-1, keepdim=True) if norm == "layer" else 0.0
        rstd = 1.0 if norm == "none" else ((x - mean).square().mean(-1, keepdim=True) + EPS) ** -0.5
        xh = (x - mean) * rstd
        w = 1.0 if gamma is None else gamma.double()
        if case["op"] == "rope":
            out[name] = _rotated(xh * w + (0.0 if beta is None else beta.double()), rot)
            continue
        dz = _rotated(s["d" + name].double(), rot, back=True)
        if norm == "none":
            out[name] = dz
            continue
        d = dz * w
        out[name] = rstd * (d - (d.mean(-1, keepdim=True) if norm == "layer" else 0.0) - xh * (d * xh).mean(-1, keepdim=True))
        out[name + "_gamma"] = torch.einsum("thd,thd->d", dz, xh)
        out[name + "_beta"] = dz.sum((0, 1)) if norm == "layer" else None
    return out


def _exact_write(case, s, cache, scale, x):
    """Cache and scales in 64 bits after x was written, one page after another."""
    held = cache.double() * scale.double()[:, :, None, None]
    unit = scale.double()
    page, most = case["page"], LARGEST[case["code"]]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    cu = list(range(case["batch"] + 1)) if s["cu"] is None else s["cu"].tolist()

    def nearest(v, u):  # to a code of unit u, in units
        v = v / u
        if case["code"] == "int8":
            return torch.round(v).clamp(-most, most)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(v / step) * step).clamp(-most, most)

    for b in range(case["batch"]):
        n = cu[b + 1] - cu[b]
        begin = lens[b] - n
        at = max(begin, 0)
        while at < lens[b]:
            end = min(lens[b], (at // page + 1) * page)
            p, lo = table[b][at // page], at % page
            new = x[cu[b] + at - begin:cu[b] + end - begin].double().transpose(0, 1)
            big = new.abs().amax((1, 2))
            u = torch.exp2(torch.round(torch.log2(big / most)).clamp(-125, 119))
            u = torch.where(big > most * u, 2 * u, torch.where(big <= most * u / 2, u / 2, u))
            if lo:
                u = torch.maximum(u, unit[p])
                held[p, :, :lo] = nearest(held[p, :, :lo], u[:, None, None]) * u[:, None, None]
            held[p, :, lo:lo + end - at] = nearest(new, u[:, None, None]) * u[:, None, None]
            unit[p] = u
            at = end
    return held, unit


def _exact_read(case, s, held):
    out = torch.zeros((case["batch"], case["longest"], case["kv_heads"], case["dim"]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n:
            pages = s["table"][b, :-(-n // case["page"])].long()
            out[b, :n] = held[pages].transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])[:n]
    return out


def _exact_attend(case, s):
    h, d, group = case["kv_heads"], case["dim"], case["group"]
    n = s["q"].shape[0]
    out = torch.zeros((n, h, group, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n, h, group), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(n, h, group, d) / math.sqrt(d)
    cu = list(range(case["batch"] + 1)) if s["cu"] is None else s["cu"].tolist()
    for b, length in enumerate(s["lens"].tolist()):
        if not length:
            continue
        pages = s["table"][b, :-(-length // case["page"])].long()
        k, v = ((s[x + "_cache"][pages].double() * s[x + "_scale"][pages].double()[:, :, None, None]).transpose(0, 1)
                .reshape(h, -1, d)[:, :length] for x in "kv")
        for i in range(cu[b], cu[b + 1]):
            seen = length - (cu[b + 1] - 1 - i)
            if s["select"] is None:
                ids = slice(0, seen)
            else:
                ids = s["select"][i].long()
                ids = ids[(ids >= 0) & (ids < seen)]
            y = torch.matmul(q[i], k[:, ids].transpose(1, 2))
            if y.shape[-1]:
                lse[i] = torch.logsumexp(y, -1)
                out[i] = torch.matmul(torch.softmax(y, -1), v[:, ids])
    return out.view(n, h * group, d), lse.view(n, h * group)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "rope_bwd"):
        return _exact_rope(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "read":
        return _exact_read(case, s, s["k_cache"].double() * s["k_scale"].double()[:, :, None, None])
    out = []
    for x in ("k", "v"):
        if s[x] is not None:
            held, unit = _exact_write(case, s, s[x + "_cache"], s[x + "_scale"], s[x])
            out += [_exact_read(case, s, held), unit]
    return out
