"""Cases of the operators that stand around the indexer's backward pass when a
model with sparse attention is trained: the layer norm of the indexer's keys
(and of hidden states) with its backward pass, the log probabilities, entropy
and top alternatives of a model's logits with their backward pass, and the
distillation of a student from a teacher's top logits with its gradient.

Each case is one call as a training loop or a sampler makes it; `run` computes
it in elementary torch operations, or through this package where `own` is set.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # keys of the tokens of one decoding step: 8 sequences, one indexer head of 128; latency alone
        dict(name="norm_step", op="norm", rows=8, width=128, type="bf16", dy="bf16", pad=0),
        # dK (fp32) of the anchor's 4096 keys back through the key norm, dx for the projection's backward
        dict(name="norm_keys_bwd", op="norm_bwd", rows=4096, width=128, type="bf16", dy="fp32", pad=0),
        # hidden states of 8192 tokens, forward and backward
        dict(name="norm_hidden", op="norm", rows=8192, width=4096, type="bf16", dy="bf16", pad=0),
        dict(name="norm_hidden_bwd", op="norm_bwd", rows=8192, width=4096, type="bf16", dy="bf16", pad=0),
        # an odd width that is a slice of a wider buffer, in fp32: no row but the first is 16-byte aligned
        dict(name="norm_odd_bwd", op="norm_bwd", rows=5003, width=2047, type="fp32", dy="fp32", pad=64),
        # the sampled tokens of one decoding step with 20 alternatives
        dict(name="logp_step", op="logp", rows=8, vocab=65536, type="bf16", top=20, temperature=1.0, masked=0.0, pad=0),
        # a teacher's pass over 2048 positions that keeps its 64 top logits
        dict(name="logp_teacher", op="logp", rows=2048, vocab=131072, type="bf16", top=64, temperature=1.0, masked=0.0, pad=0),
        # odd vocabulary in padded rows, a third of it masked out, sampling temperature
        dict(name="logp_masked", op="logp", rows=1021, vocab=50001, type="fp32", top=8, temperature=0.7, masked=0.3, pad=47),
        # policy gradient with an entropy bonus
        dict(name="logp_bwd", op="logp_bwd", rows=2048, vocab=65536, type="bf16", temperature=1.0, pad=0),
        # a short sequence's loss and gradient
        dict(name="distill_short", op="distill", rows=32, vocab=32768, type="bf16", top=32, temperature=1.0, pad=0),
        # a training batch of 4096 tokens: loss and gradient in one call
        dict(name="distill_batch", op="distill", rows=4096, vocab=131072, type="bf16", top=64, temperature=1.0, pad=0),
        # loss first, gradient when its own upstream gradient is known; odd vocabulary, softened targets
        dict(name="distill_split", op="distill_split", rows=1023, vocab=50001, type="fp16", top=100, temperature=2.0, pad=0),
    ]


def _size(rng, lo, hi, multiple=1):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, n // multiple * multiple)
    return n + multiple if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "logp", "logp_bwd", "distill", "distill_split"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_bwd"):
        width = _size(rng, 32, 16384, rng.choice([1, 8, 128 if rng.random() < 0.5 else 64]))
        rows = _size(rng, 1, min(32768, (1 << 26) // width))
        dy = rng.choice([kind, "fp32"])
        pad = rng.choice([0, 0, 8, 5])
        return dict(op=op, rows=rows, width=width, type=kind, dy=dy, pad=0 if width + pad == 3072 else pad)
    vocab = _size(rng, 1000, 131072, rng.choice([1, 8, 256]))
    rows = _size(rng, 1, min(8192, (1 << 28) // vocab))
    case = dict(op=op, rows=rows, vocab=vocab, type=kind, temperature=rng.choice([1.0, 1.0, 0.7, 2.0]),
                pad=rng.choice([0, 0, 8, 3]))
    if op == "logp":
        case.update(top=rng.choice([0, 1, 5, 20, 64, 128]), masked=rng.choice([0.0, 0.0, 0.3, 0.9]))
    elif op != "logp_bwd":
        case.update(top=rng.choice([1, 8, 32, 100, 256]))
    return case


def _normal(g, rows, width, pad):
    """Normal values in a buffer of width + pad columns, of which a case takes the first `width`."""
    x = torch.empty((rows, width + pad), dtype=torch.float32, device="cuda")
    x.normal_(generator=g)
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = TYPES[case["type"]]
    rows, pad = case["rows"], case["pad"]
    s = dict(case=case)
    if case["op"] in ("norm", "norm_bwd"):
        n = case["width"]
        x = _normal(g, rows, n, pad)
        # rows of different size and offset, as a projection gives them
        x.mul_(torch.rand((rows, 1), device="cuda", generator=g) * 2 + 0.25)
        x.add_(torch.randn((rows, 1), device="cuda", generator=g) * 0.5)
        s["x"] = x.to(dt)[:, :n]
        s["gamma"] = 1 + 0.2 * torch.randn(n, device="cuda", generator=g)
        s["beta"] = 0.2 * torch.randn(n, device="cuda", generator=g)
        if case["op"] == "norm_bwd":
            s["dy"] = _normal(g, rows, n, pad).to(TYPES[case["dy"]])[:, :n]
            xs = s["x"].double()
            s["mean"] = xs.mean(1).float()
            s["rstd"] = (xs.var(1, unbiased=False) + EPS).rsqrt().float()
        return s
    v = case["vocab"]
    x = _normal(g, rows, v, pad).mul_(2.5)
    # a few likely tokens in each row, none of them twice
    tokens = torch.randint(0, v, (rows, 1), device="cuda", generator=g)
    likely = (tokens + torch.arange(16, device="cuda") * (v // 16)) % v
    x.scatter_add_(1, likely, 6 * torch.rand((rows, 16), device="cuda", generator=g))
    tokens = tokens[:, 0].to(torch.int32)
    if case["op"] == "logp" and case["masked"] > 0:
        keep = torch.rand((1, v), device="cuda", generator=g) >= case["masked"]
        keep[:, 0] = True
        x[:, :v].masked_fill_(~keep, -math.inf)
    s["logits"] = x.to(dt)[:, :v]
    if case["op"] in ("logp", "logp_bwd"):
        s["tokens"] = tokens
    if case["op"] == "logp_bwd":
        y = s["logits"].float() / case["temperature"]
        s["lse"] = torch.logsumexp(y, 1)
        p = torch.exp(y - s["lse"][:, None])
        s["entropy"] = s["lse"] - (p * y).sum(1)
        scale = (4096 if dt == torch.float16 else 1) / rows  # a gradient in fp16 carries a loss scale
        s["dlogprob"] = torch.randn(rows, device="cuda", generator=g) * scale
        s["dentropy"] = torch.full((rows,), -0.01 * scale, device="cuda")
    if case["op"] in ("distill", "distill_split"):
        k = min(case["top"], v)
        # the teacher agrees with the student up to noise; its top tokens, best first
        t = x[:, :v] + torch.randn((rows, 1), device="cuda", generator=g)
        t += 0.7 * torch.randn((1, v), device="cuda", generator=g)
        val, ids = torch.topk(t, k, dim=1)
        s["teacher"] = val.contiguous()
        s["ids"] = ids.to(torch.int32).contiguous()
        # some rows keep fewer tokens than others: -1 where nothing is left
        few = torch.randint(0, 4 * k + 1, (rows, 1), device="cuda", generator=g)
        s["ids"].masked_fill_(torch.arange(k, device="cuda")[None, :] >= few, -1)
        # prompt tokens carry no loss; a gradient in fp16 carries a loss scale
        weight = (torch.rand(rows, device="cuda", generator=g) < 0.8).float() / rows
        weight *= 4096 if dt == torch.float16 else 1
        s["weight" if case["op"] == "distill" else "dloss"] = weight
    return s


# ------------------------------------------------------------- plain forms ---

def _norm(x, gamma, beta):
    x32 = x.float()
    mean = x32.sum(1) / x.shape[1]
    d = x32 - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).sum(1) / x.shape[1] + EPS)
    y = d * rstd[:, None] * gamma + beta
    return y.to(x.dtype), mean, rstd


def _norm_bwd(dy, x, mean, rstd, gamma):
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    d32 = dy.float()
    d = d32 * gamma
    n = x.shape[1]
    dx = rstd[:, None] * (d - d.sum(1, keepdim=True) / n - xh * ((d * xh).sum(1, keepdim=True) / n))
    return dx.to(x.dtype), (d32 * xh).sum(0), d32.sum(0)


def _softmax_stats(y):
    m = y.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    d = y - m
    e = torch.exp(d)
    z = e.sum(1, keepdim=True)
    return m, d, e, z


def _logp(x, tokens, top, temperature):
    x32 = x.float()
    y = x32 / temperature
    m, d, e, z = _softmax_stats(y)
    lz = torch.log(z)
    entropy = (lz - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1, keepdim=True) / z)[:, 0]
    lse = (m + lz)[:, 0]
    logprob = d.gather(1, tokens.long()[:, None])[:, 0] - lz[:, 0]
    if not top:
        return logprob, entropy, lse
    # order by value, then by lowest index: one whole number for each entry
    n = min(top, x.shape[1])
    bits = (x32 + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
    key = key * (1 << 32) + torch.arange(x.shape[1] - 1, -1, -1, device=x.device)
    ids = x.shape[1] - 1 - (torch.topk(key, n, dim=1).values & 0xFFFFFFFF)
    val = d.gather(1, ids) - lz
    return logprob, entropy, lse, torch.where(val > -math.inf, ids, torch.full_like(ids, -1)).to(torch.int32), val


def _logp_bwd(x, tokens, lse, entropy, dlogprob, dentropy, temperature):
    y = x.float() / temperature
    lp = y - lse[:, None]
    q = torch.exp(lp)
    g = -q * (dlogprob[:, None] + dentropy[:, None] * torch.where(q > 0, lp + entropy[:, None], torch.zeros_like(lp)))
    g.scatter_add_(1, tokens.long()[:, None], dlogprob[:, None])
    return (g / temperature).to(x.dtype)


def _targets(ids, teacher, temperature):
    """The teacher's probabilities over its kept tokens, and their logarithms."""
    ok = ids >= 0
    t = torch.where(ok, teacher / temperature, torch.full_like(teacher, -math.inf))
    m, d, e, z = _softmax_stats(t)
    any_ = z > 0
    p = torch.where(any_, e / torch.where(any_, z, torch.ones_like(z)), torch.zeros_like(e))
    return p, d - torch.log(z), torch.where(ok, ids, torch.zeros_like(ids)).long(), any_


def _distill_loss(y, lse, ids, teacher, temperature):
    p, logp, at, any_ = _targets(ids, teacher, temperature)
    gap = logp - (y.gather(1, at) - lse[:, None])
    loss = temperature * temperature * torch.where(p > 0, p * gap, torch.zeros_like(p)).sum(1)
    return loss, p, at, any_


def _distill_grad(y, lse, p, at, any_, scale, temperature):
    g = torch.exp(y - lse[:, None])
    g = torch.where(any_, g, torch.zeros_like(g))
    g.scatter_add_(1, at, -p)
    return g * (scale * temperature)[:, None]


def _lse(y):
    m, d, e, z = _softmax_stats(y)
    return (m + torch.log(z))[:, 0]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        return _norm(s["x"], s["gamma"], s["beta"])
    if op == "norm_bwd":
        return _norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"])
    if op == "logp":
        return _logp(s["logits"], s["tokens"], c["top"], c["temperature"])
    if op == "logp_bwd":
        return _logp_bwd(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogprob"], s["dentropy"],
                         c["temperature"])
    y = s["logits"].float() / c["temperature"]
    lse = _lse(y)
    loss, p, at, any_ = _distill_loss(y, lse, s["ids"], s["teacher"], c["temperature"])
    if op == "distill":
        dx = _distill_grad(y, lse, p, at, any_, s["weight"], c["temperature"])
        return loss, dx.to(s["logits"].dtype)
    dx = _distill_grad(y, lse, p, at, any_, s["dloss"], c["temperature"])
    return loss, lse, dx.to(s["logits"].dtype)


def _own(s):
    import sparse_attention_indexer_bwd_gb300 as ibwd
    c = s["case"]
    op = c["op"]
    if op == "norm":
        return ibwd.layer_norm_fwd(s["x"], s["gamma"], s["beta"], eps=EPS)
    if op == "norm_bwd":
        return ibwd.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"])
    if op == "logp":
        n = min(c["top"], c["vocab"])
        out = ibwd.token_logprobs_fwd(s["logits"], s["tokens"], top_n=n, temperature=c["temperature"])
        return out if n else out[:3]
    if op == "logp_bwd":
        return ibwd.token_logprobs_bwd(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogprob"],
                                       s["dentropy"], temperature=c["temperature"])
    if op == "distill":
        return ibwd.distill_grad(s["logits"], s["ids"], s["teacher"], s["weight"], temperature=c["temperature"])
    loss, lse = ibwd.distill_fwd(s["logits"], s["ids"], s["teacher"], temperature=c["temperature"])
    dx = ibwd.distill_bwd(s["logits"], s["ids"], s["teacher"], lse, s["dloss"], temperature=c["temperature"])
    return loss, lse, dx


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------- work and 64-bit results ---

def work(case):
    size = {"fp32": 4, "bf16": 2, "fp16": 2}
    rows, e = case["rows"], size[case["type"]]
    if case["op"] == "norm":
        n = case["width"]
        return {"bytes": rows * n * 2 * e + 8 * n + 8 * rows, "flops": 8 * rows * n}
    if case["op"] == "norm_bwd":
        n = case["width"]
        return {"bytes": rows * n * (2 * e + size[case["dy"]]) + 12 * n + 8 * rows, "flops": 14 * rows * n}
    v = case["vocab"]
    if case["op"] == "logp":
        return {"bytes": rows * v * e + rows * (4 + 12 + 8 * case["top"]), "flops": 6 * rows * v}
    if case["op"] == "logp_bwd":
        return {"bytes": rows * v * 2 * e + rows * 20, "flops": 8 * rows * v}
    passes = 2 if case["op"] == "distill" else 3  # the split form has to read the logits twice
    return {"bytes": rows * v * passes * e + rows * (8 * case["top"] + 12), "flops": 8 * rows * v}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        mean = x.mean(1)
        var = x.var(1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * s["gamma"].double() + s["beta"].double()
        return y, mean, rstd
    if op == "norm_bwd":
        x, dy, w = s["x"].double(), s["dy"].double(), s["gamma"].double()
        n = x.shape[1]
        xh = (x - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        d = dy * w
        a, b = d.mean(1), (d * xh).mean(1)
        return ((d - a[:, None] - b[:, None] * xh) * s["rstd"].double()[:, None],
                torch.einsum("rn,rn->n", dy, xh), dy.sum(0))
    rows, v, tau = case["rows"], case["vocab"], case["temperature"]
    parts = []
    step = max(1, (1 << 25) // v)
    for a in range(0, rows, step):
        r = slice(a, min(rows, a + step))
        x = s["logits"][r].double()
        lp = torch.log_softmax(x / tau, 1)
        q = lp.exp()
        if op == "logp":
            h = torch.special.entr(q).sum(1)
            out = [lp.gather(1, s["tokens"][r].long()[:, None])[:, 0], h, torch.logsumexp(x / tau, 1)]
            if case["top"]:
                ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :min(case["top"], v)]
                best = lp.gather(1, ids)
                out += [torch.where(best == -math.inf, -1, ids).to(torch.int32), best]
        elif op == "logp_bwd":
            # d(logprob) = onehot - q; d(entropy) = -q (log q + entropy); the statistics are given
            lp = x / tau - s["lse"][r].double()[:, None]
            q = lp.exp()
            hot = torch.zeros_like(q)
            hot[torch.arange(hot.shape[0], device=hot.device), s["tokens"][r].long()] = 1
            g = s["dlogprob"][r].double()[:, None] * (hot - q)
            g -= s["dentropy"][r].double()[:, None] * q * (lp + s["entropy"][r].double()[:, None])
            out = [g / tau]
        else:
            ids, t = s["ids"][r].long(), s["teacher"][r].double()
            p = torch.zeros((ids.shape[0], v + 1), dtype=torch.float64, device=x.device)
            at = torch.where(ids < 0, v, ids)
            t = torch.where(ids < 0, -math.inf, t / tau)
            p.scatter_(1, at, torch.softmax(t, 1))
            p = p[:, :v]
            loss = tau * tau * torch.where(p > 0, p * (p.log() - lp), 0.0).sum(1)
            w = s["weight" if op == "distill" else "dloss"][r].double()
            w = torch.where((ids >= 0).any(1), w, 0.0)  # a row that keeps no token has no target
            g = tau * w[:, None] * (q - p)
            out = [loss, g] if op == "distill" else [loss, torch.logsumexp(x / tau, 1), g]
        parts.append(out)
    got = [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]))]
    return got[0] if op == "logp_bwd" else got
