"""Token log probabilities and distillation, forward and backward, against
plain 64-bit forms."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from train_ref import (DTYPES, U, check_distill, check_logp_bwd, check_logp_fwd, distill, logp_fwd)

pytestmark = pytest.mark.gpu

INF = math.inf


def logits(rows, v, kind="bf16", pad=0, offset=0, seed=0, size=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(rows * (v + pad) + offset, device="cuda", generator=g) * size
    buf += 5 * (torch.rand(buf.shape, device="cuda", generator=g) < 0.001)
    return buf.to(DTYPES[kind])[offset:].view(rows, v + pad)[:, :v]


def some_tokens(rows, v, seed=1, padding=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, v, (rows,), device="cuda", generator=g, dtype=torch.int32)
    if padding and rows > 2:
        t[1], t[2] = -100, v
    return t


def kept(x, k, seed=2, padding=True):
    """Teacher's ids and values for logits x: the student's top tokens moved by noise, some slots padding."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.where(torch.isfinite(x.float()), x.float(), -30.0)
    t = t + torch.randn(x.shape, device="cuda", generator=g)
    val, ids = torch.topk(t, k, dim=1)
    ids = ids.to(torch.int32)
    if padding:
        drop = torch.rand(ids.shape, device="cuda", generator=g) < 0.2
        ids = torch.where(drop, torch.where(val > 2, -1, x.shape[1] + 5).to(torch.int32), ids)
        val = torch.where(drop, torch.where(ids < 0, math.nan, 1e30), val)
    return ids, val


def same(a, b):
    if a is None:
        return b is None
    view = {4: torch.int32, 2: torch.int16}
    return torch.equal(a.contiguous().view(view[a.element_size()]), b.contiguous().view(view[b.element_size()]))


def check_all(x, tau, top, k, what, tokens=None):
    rows, v = x.shape
    tokens = some_tokens(rows, v) if tokens is None else tokens
    got = ibwd.token_logprobs_fwd(x, tokens, top_n=top, temperature=tau)
    check_logp_fwd(got, x, tokens, top, tau, what)
    g = torch.Generator(device="cuda").manual_seed(3)
    da, dh = torch.randn(rows, device="cuda", generator=g), torch.randn(rows, device="cuda", generator=g)
    _, entropy, lse = got[:3]
    fine = torch.isfinite(entropy)
    for a, h in ((da, dh), (da, None), (None, dh)):
        dx = ibwd.token_logprobs_bwd(x, tokens, lse, entropy, a, h, temperature=tau)
        pick = [None if t is None else t[fine] for t in (tokens, lse, entropy, a, h)]
        check_logp_bwd(dx[fine], x[fine], *pick, tau, what + " bwd")
    ids, teacher = kept(x, k)
    w = torch.rand(rows, device="cuda", generator=g)
    loss, lse2 = ibwd.distill_fwd(x, ids, teacher, temperature=tau)
    dx = ibwd.distill_bwd(x, ids, teacher, lse2, w, temperature=tau)
    check_distill(loss, lse2, dx, w, x, ids, teacher, tau, what + " split")
    loss3, dx3 = ibwd.distill_grad(x, ids, teacher, w, grad_scale=0.5, temperature=tau)
    check_distill(loss3, None, dx3, 0.5 * w, x, ids, teacher, tau, what + " whole")


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("v", [1, 2, 7, 8, 63, 100, 513, 1000, 4097, 8192, 12345])
def test_vocabularies(v, kind):
    for rows in (1, 9):
        check_all(logits(rows, v, kind, seed=v), 1.0, min(v, 5), min(v, 7), f"{rows}x{v}")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,v", [(1, 50001), (3, 131072), (17, 65536), (40, 131071), (80, 32768), (160, 50001),
                                    (400, 32000), (2, 300001)])
def test_few_and_many_rows(rows, v, kind):
    """From one row, which a cluster of blocks shares, to one block a row."""
    check_all(logits(rows, v, kind, seed=rows), 0.7, 20, 64, f"{rows}x{v}")


@pytest.mark.parametrize("top", [1, 2, 64, 127, 128])
@pytest.mark.parametrize("rows,v", [(2, 128), (2, 40000), (310, 5000)])
def test_numbers_of_alternatives(rows, v, top):
    for kind in ("bf16", "fp32"):
        check_logp_fwd(ibwd.token_logprobs_fwd(x := logits(rows, v, kind, seed=top), None, top_n=top), x, None, top, 1.0,
                       f"top {top}")


@pytest.mark.parametrize("k", [1, 3, 128, 513, 1024])
def test_numbers_of_kept_tokens(k):
    for rows, v in ((2, 40000), (310, 2000)):
        x = logits(rows, v, "fp32", seed=k)
        ids, teacher = kept(x, k)
        w = torch.ones(rows, device="cuda")
        loss, dx = ibwd.distill_grad(x, ids, teacher)
        check_distill(loss, None, dx, w, x, ids, teacher, 1.0, f"K {k}")


@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (8, 1), (0, 3), (5, 7)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_strides_and_alignments(pad, offset, kind):
    for rows, v in ((3, 40007), (330, 1001)):
        x = logits(rows, v, kind, pad, offset, seed=5)
        check_all(x, 1.3, 8, 16, f"pad {pad} offset {offset}")
        ids, teacher = kept(x, 16)
        buf = torch.full((rows, v + 6), 7.0, device="cuda", dtype=x.dtype)  # another row alignment than the logits
        loss, dx = ibwd.distill_grad(x, ids, teacher, out=buf[:, :v])
        check_distill(loss, None, dx, torch.ones(rows, device="cuda"), x, ids, teacher, 1.0, "strided out")
        assert (buf[:, v:] == 7).all()
        dx = ibwd.distill_grad(x, ids, teacher)[1]
        assert dx.stride() == x.stride()
        assert same(dx, buf[:, :v])


@pytest.mark.parametrize("rows,v", [(4, 70000), (330, 3001)])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_masked_logits(rows, v, kind):
    """Masks of -inf and of the type's lowest value, rows of one token and of none."""
    low = torch.finfo(DTYPES[kind]).min
    for fill in (-INF, low):
        x = logits(rows, v, kind, seed=6)
        x[torch.rand(x.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)) < 0.999] = fill
        x[0] = fill
        x[1] = fill
        x[1, v - 1] = 1.5
        got = ibwd.token_logprobs_fwd(x, some_tokens(rows, v, padding=False), top_n=30)
        check_logp_fwd(got, x, some_tokens(rows, v, padding=False), 30, 1.0, f"masked {fill}")
        if fill == -INF:
            assert got[2][0] == -INF and got[1][0] == 0 and got[0][0] == -INF and (got[3][0] == -1).all()
            check_all(x, 1.0, 30, 8, "masked")
            ones = torch.ones(rows, device="cuda")
            tok = some_tokens(rows, v, padding=False)
            assert (ibwd.token_logprobs_bwd(x, tok, got[2], got[1], ones, ones)[0] == 0).all()
            ids, teacher = kept(x, 8)
            loss, dx = ibwd.distill_grad(x, ids, teacher)
            assert loss[0] == 0 and (dx[0] == 0).all()
        else:
            # the whole row at the lowest value is a uniform row
            assert abs(got[1][0].item() - math.log(v)) < 1e-4
            assert torch.equal(got[3][0].cpu(), torch.arange(30, dtype=torch.int32))
            ids, teacher = kept(x, 8, padding=False)
            loss, dx = ibwd.distill_grad(x, ids, teacher)
            check_distill(None, None, dx, torch.ones(rows, device="cuda"), x, ids, teacher, 1.0, "lowest")


@pytest.mark.parametrize("rows", [2, 320])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_ties_and_orders_of_the_top(rows, kind):
    """Equal logits, sorted logits and logits whose size follows the threads that read them."""
    v = 40960
    at = torch.arange(v, device="cuda")
    patterns = {
        "equal": torch.zeros(v, device="cuda"),
        "zeros of both signs": torch.where(at % 3 == 0, -0.0, 0.0),
        "rising": at / 64.0,
        "falling": -at / 64.0,
        "two values": (at % 7 == 3).float(),
        "few high": torch.where(at % 4096 == 5, 3.0, 1.0),
        "threads": torch.where((at // 8) % 512 < 64, 100.0 + (at % 4099) / 256, 0.0),
        "threads of four": torch.where((at // 4) % 512 < 100, 100.0 + (at % 4099) / 256, 0.0),
        "one block": torch.where(at < 3000, 50.0 + (at % 977) / 64, 0.0),
        "mostly masked": torch.where(at % 1000 == 1, at / 4096.0, -INF),
    }
    for name, p in patterns.items():
        x = p.to(DTYPES[kind]).expand(rows, v).contiguous()
        for top in (1, 64, 128):
            got = ibwd.token_logprobs_fwd(x, None, top_n=top)
            check_logp_fwd(got, x, None, top, 1.0, f"{name} top {top}")


def test_nan_and_infinity():
    for rows, v in ((4, 50000), (310, 1000)):
        x = logits(rows, v, "fp32", seed=8)
        clean = ibwd.token_logprobs_fwd(x, some_tokens(rows, v), top_n=9)
        x[0, 17] = math.nan
        x[1, v - 3] = INF
        x[3] = -INF
        x[3, 2] = math.nan
        tok = some_tokens(rows, v)
        got = ibwd.token_logprobs_fwd(x, tok, top_n=9)
        check_logp_fwd(got, x, tok, 9, 1.0, "NaN")
        for a, b in zip(got, clean):
            assert same(a[4:], b[4:]) and same(a[2:3], b[2:3])
        ids, teacher = kept(x, 8, padding=False)
        loss, dx = ibwd.distill_grad(x, ids, teacher)
        assert torch.isnan(loss[[0, 1, 3]]).all() and torch.isfinite(loss[2]) and torch.isfinite(dx[2]).all()
        assert torch.isnan(dx[0]).all()


def test_teacher_slots():
    """Repeated tokens, rows that keep nothing, slots of -inf, a kept token that the student masks."""
    for rows, v in ((6, 40000), (320, 999)):
        x = logits(rows, v, "fp32", seed=9)
        ids, teacher = kept(x, 12, padding=False)
        ids[0] = ids[0, 3]                       # one token in every slot
        ids[1, ::2] = ids[1, 1]
        ids[2] = -1                              # nothing kept
        teacher[3] = -INF                        # kept, but without mass
        teacher[4, 5:] = -INF
        w = torch.ones(rows, device="cuda")
        loss, lse = ibwd.distill_fwd(x, ids, teacher, temperature=2.0)
        dx = ibwd.distill_bwd(x, ids, teacher, lse, w, temperature=2.0)
        check_distill(loss, lse, dx, w, x, ids, teacher, 2.0, "slots")
        whole = ibwd.distill_grad(x, ids, teacher, temperature=2.0)
        check_distill(whole[0], None, whole[1], w, x, ids, teacher, 2.0, "slots, whole")
        assert loss[2] == 0 and loss[3] == 0 and (dx[2:4] == 0).all() and (whole[1][2:4] == 0).all()
        x[5, ids[5, 0].long()] = -INF
        loss, dx = ibwd.distill_grad(x, ids, teacher, temperature=2.0)
        assert loss[5] == INF and torch.isfinite(dx).all()
        check_distill(loss, None, dx, w, x, ids, teacher, 2.0, "masked by the student")


@pytest.mark.parametrize("rows,v", [(3, 70001), (3, 65536), (310, 3001)])
def test_in_place_and_reproducible(rows, v):
    for kind in ("bf16", "fp32"):
        x = logits(rows, v, kind, seed=10)
        tok = some_tokens(rows, v)
        ids, teacher = kept(x, 40)
        got = ibwd.token_logprobs_fwd(x, tok, top_n=33)
        a = torch.rand(rows, device="cuda")
        dx = ibwd.token_logprobs_bwd(x, tok, got[2], got[1], a, a)
        split = ibwd.distill_bwd(x, ids, teacher, got[2], a)
        loss, whole = ibwd.distill_grad(x, ids, teacher, a)
        for _ in range(3):
            again = ibwd.token_logprobs_fwd(x, tok, top_n=33)
            assert all(same(p, q) for p, q in zip(got, again))
            l2, w2 = ibwd.distill_grad(x, ids, teacher, a)
            assert same(l2, loss) and same(w2, whole)
        z = x.clone()
        assert ibwd.token_logprobs_bwd(z, tok, got[2], got[1], a, a, out=z) is z and same(z, dx)
        z = x.clone()
        assert same(ibwd.distill_bwd(z, ids, teacher, got[2], a, out=z), split)
        z = x.clone()
        l2, w2 = ibwd.distill_grad(z, ids, teacher, a, out=z)
        assert w2 is z and same(l2, loss) and same(z, whole)


def test_no_rows_and_leading_dimensions():
    x = torch.empty((0, 1000), device="cuda")
    e = torch.empty((0,), device="cuda")
    ids = torch.empty((0, 4), device="cuda", dtype=torch.int32)
    assert ibwd.token_logprobs_fwd(x, e.to(torch.int32), top_n=3)[4].shape == (0, 3)
    assert ibwd.token_logprobs_bwd(x, None, e, e, None, e).shape == (0, 1000)
    assert ibwd.distill_grad(x, ids, ids.float())[1].shape == (0, 1000)
    x = logits(6, 999, "bf16").view(2, 3, 999)
    tok = some_tokens(6, 999).view(2, 3)
    a, b = ibwd.token_logprobs_fwd(x, tok, top_n=4), ibwd.token_logprobs_fwd(x.view(6, 999), tok.view(6), top_n=4)
    assert a[4].shape == (2, 3, 4) and all(same(p.flatten(), q.flatten()) for p, q in zip(a, b))
    ids, teacher = kept(x.view(6, 999), 5)
    loss, dx = ibwd.distill_grad(x, ids.view(2, 3, 5), teacher.view(2, 3, 5))
    assert loss.shape == (2, 3) and dx.shape == x.shape
    assert same(dx.view(6, 999), ibwd.distill_grad(x.view(6, 999), ids, teacher)[1])


def test_gradients_against_differences():
    """The gradients against central differences of the 64-bit losses."""
    x = logits(3, 37, "fp32", seed=11, size=1.0)
    tok = some_tokens(3, 37, padding=False)
    a, h = torch.rand(3, device="cuda"), torch.rand(3, device="cuda")
    ids, teacher = kept(x, 6)
    teacher = torch.where(torch.isfinite(teacher), teacher, 0.0)
    tau, step = 1.5, 1e-5
    got = ibwd.token_logprobs_fwd(x, tok, temperature=tau)
    d1 = ibwd.token_logprobs_bwd(x, tok, got[2], got[1], a, h, temperature=tau)
    _, d2 = ibwd.distill_grad(x, ids, teacher, a, grad_scale=2.0, temperature=tau)

    def f1(y):
        lp, e, _ = logp_fwd(y, tok, 0, tau)
        return (lp * a.double() + e * h.double()).sum()

    def f2(y):
        return 2 * (distill(y, ids, teacher, tau)[0] * a.double()).sum()

    y = x.double()
    for i in range(0, y.numel(), 2):
        flat = y.view(-1)
        keep = flat[i].clone()
        for f, d in ((f1, d1), (f2, d2)):
            flat[i] = keep + step
            up = f(y)
            flat[i] = keep - step
            down = f(y)
            flat[i] = keep
            assert abs((up - down) / (2 * step) - d.view(-1)[i]) < 1e-6


def test_other_stream_and_graph():
    x = logits(5, 60000, "bf16", seed=12)
    tok = some_tokens(5, 60000)
    ids, teacher = kept(x, 16)
    want = ibwd.token_logprobs_fwd(x, tok, top_n=10)
    wl, wd = ibwd.distill_grad(x, ids, teacher)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ibwd.token_logprobs_fwd(x, tok, top_n=10, stream=s)
    l2, d2 = ibwd.distill_grad(x, ids, teacher, stream=s.cuda_stream)
    s.synchronize()
    assert all(same(p, q) for p, q in zip(want, got)) and same(l2, wl) and same(d2, wd)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = ibwd.token_logprobs_fwd(x, tok, top_n=10)
        l3, d3 = ibwd.distill_grad(x, ids, teacher)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(same(p, q) for p, q in zip(want, got)) and same(l3, wl) and same(d3, wd)


def test_offsets_past_32_bits():
    """Rows beyond 2^32 elements: first and last rows against the same rows alone."""
    v, rows = 131072, 33000
    x = torch.empty((rows, v), device="cuda", dtype=torch.bfloat16)
    x.fill_(-4)
    some = torch.tensor([0, 1, 16383, 16384, 32767, 32768, rows - 1], device="cuda")
    x[some] = logits(len(some), v, "bf16", seed=13)
    tok = some_tokens(rows, v, padding=False)
    ids = torch.zeros((rows, 4), device="cuda", dtype=torch.int32)
    teacher = torch.zeros((rows, 4), device="cuda")
    ids[some], teacher[some] = kept(x[some], 4)
    got = ibwd.token_logprobs_fwd(x, tok, top_n=5)
    check_logp_fwd([t[some] for t in got], x[some], tok[some], 5, 1.0, "far rows")
    part = x[some]
    loss, dx = ibwd.distill_grad(x, ids, teacher, out=x)
    check_distill(loss[some], None, dx[some], torch.ones(len(some), device="cuda"), part, ids[some], teacher[some], 1.0,
                  "far rows")


@pytest.mark.parametrize("rows,v,kind", [(2, 400000, "bf16"), (3, 170001, "fp32"), (700, 9000, "bf16"), (500, 18001, "fp16"),
                                         (200, 37000, "bf16"), (170, 70001, "bf16"), (90, 150000, "bf16"),
                                         (160, 60000, "fp32")])
def test_loss_and_gradient_over_row_sizes(rows, v, kind):
    """Rows that fit one, several or no blocks' shared memory, several rows a block."""
    x = logits(rows, v, kind, seed=rows)
    ids, teacher = kept(x, 30)
    w = torch.rand(rows, device="cuda")
    loss, dx = ibwd.distill_grad(x, ids, teacher, w)
    step = max(1, (1 << 23) // v)
    for a in range(0, rows, step):
        r = slice(a, min(rows, a + step))
        check_distill(loss[r], None, dx[r], w[r], x[r], ids[r], teacher[r], 1.0, f"{rows}x{v}")
    z = x.clone()
    l2, d2 = ibwd.distill_grad(z, ids, teacher, w, out=z)
    assert same(l2, loss) and same(z, dx)


@pytest.mark.parametrize("tau", [1e-7, 1e-3, 50.0, 1e4, 1e21])
@pytest.mark.parametrize("kind", ["fp16", "fp32"])
def test_extreme_temperatures(tau, kind):
    """From an argmax to a uniform row, with masks of -inf and of the lowest value."""
    for rows, v in ((3, 40001), (320, 1500)):
        x = logits(rows, v, kind, seed=14)
        x[:, ::3] = -INF
        x[:, 1::7] = torch.finfo(x.dtype).min
        tok = some_tokens(rows, v, padding=False)
        got = ibwd.token_logprobs_fwd(x, tok, top_n=9, temperature=tau)
        assert not any(torch.isnan(t.float()).any() for t in got)
        check_logp_fwd(got, x, tok, 9, tau, f"temperature {tau}")
        ids, teacher = kept(x, 12, padding=False)
        w = torch.ones(rows, device="cuda")
        loss, lse = ibwd.distill_fwd(x, ids, teacher, temperature=tau)
        dx = ibwd.distill_bwd(x, ids, teacher, lse, w, temperature=tau)
        whole = ibwd.distill_grad(x, ids, teacher, temperature=tau)
        # (a gradient of T (q - p) may pass the type's range, a NaN it never is)
        assert not torch.isnan(dx).any() and not torch.isnan(whole[1]).any()
        if tau >= 1e-3:
            check_distill(loss, lse, dx, w, x, ids, teacher, tau, f"temperature {tau}")
            check_distill(whole[0], None, whole[1], w, x, ids, teacher, tau, f"temperature {tau}, whole")
