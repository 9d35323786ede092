"""The attention over the 8-bit cache at the ends of its range: large logits, scales of any value."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from heads_ref import check_attention
from test_gpu_cache import CODES, E4M3, filled, generator, offsets, pages_for
from train_ref import U, half_step, within

pytestmark = pytest.mark.gpu


def alike(lens, dim, page, code, logit, group, kept, seed):
    """Sequences whose positions all have the logit `logit`, and values in blocks whose scales are no powers of two: the
    outputs are means. Every product of a query and a key is the same sum, whatever the order of its terms, so that the
    weights are off by their own roundings alone: fp16 (2^-11), 2^-22 an exponential, the units' and the sums' as counted
    elsewhere, however large the logit is."""
    table, pages = pages_for(lens, page, 1, seed)
    kc = torch.ones((pages, 1, page, dim), device="cuda").to(code)
    ks = torch.full((pages, 1), 1.37, device="cuda")
    vc, _ = filled(pages, 1, page, dim, code, seed)
    vs = 0.01 + 0.02 * torch.rand((pages, 1), device="cuda", generator=generator(seed + 1))
    q = torch.ones((len(lens), group, dim), device="cuda", dtype=torch.float16)
    dl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    select = None
    if kept:
        select = torch.stack([torch.randint(0, n, (kept,), device="cuda", generator=generator(seed + 2), dtype=torch.int32) for n in lens])
    out, lse = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, select=select, scale=logit / (1.37 * dim))
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda") if select is None else select[b].long()
        p = table[b].long()[at // page]
        v = vc[p, 0, at % page].float().double() * vs[p, 0].double()[:, None]
        ref, size = v.mean(0).expand(group, dim), v.abs().mean(0).expand(group, dim)
        rel = 2.0 ** -11 + 2.0 ** -19 + (len(at) / 16 + 64) * 2 * U
        within(out[b], ref, half_step(torch.float16) * ref.abs() + 2.0 ** -25 + rel * size, f"{n} positions, logit {logit}")
        # (the scale and its product with a key's are two roundings, the logarithm's two more)
        true = torch.full((group,), logit + math.log(len(at)), dtype=torch.float64)
        within(lse[b], true, 8 * U * (abs(logit) + 16) + 2.0 ** -20, f"{n} positions, logit {logit}: lse")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("logit", [0.0, 700.0, -3e5, 3e5, 2e7, -1e9])
def test_large_logits_with_scales_of_any_value(logit, dim, code):
    for group in (1, 5, 20):
        alike([1, 5, 300, 64], dim, 16, CODES[code], logit, group, 0, 1)
        alike([7, 300, 64], dim, 16, CODES[code], logit, group, 3, 2)
        alike([400, 300], dim, 32, CODES[code], logit, group, 200, 3)
    alike([9000], dim, 64, CODES[code], logit, 4, 0, 4)  # (one item in all blocks)


def of_scales(exponents, logits, dim, code, kept, kind, counts=None, seed=1):
    """One sequence, a page of 16 positions a block: 2^exponents[i] the scale of page i's values, logits[i] its logits."""
    n, page = 16 * len(exponents), 16
    table, pages = pages_for([n], page, 1, seed)
    at = table[0].long()
    kc = torch.zeros((pages, 1, page, dim), device="cuda")
    kc[at, 0, :, 0] = torch.tensor(logits, device="cuda", dtype=torch.float32)[:, None]  # (whole numbers of a few bits)
    kc, ks = kc.to(code), torch.ones((pages, 1), device="cuda")
    vc, vs = filled(pages, 1, page, dim, code, seed)
    vs[at, 0] = torch.exp2(torch.tensor(exponents, device="cuda", dtype=torch.float32))
    tokens = 1 if counts is None else sum(counts)
    q = torch.zeros((tokens, 3, dim), device="cuda", dtype=kind)
    q[..., 0] = 1
    dl = torch.tensor([n], device="cuda", dtype=torch.int32)
    select = None
    if kept:
        select = torch.randperm(n, device="cuda", generator=generator(seed + 1))[:kept].int().expand(tokens, kept).contiguous()
    cu = None if counts is None else offsets(counts)
    got = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, cu=cu, select=select, scale=1.0)
    check_attention(got, q, kc, vc, ks, vs, table, [n], None if cu is None else cu.tolist(), select, 1.0, page,
                    f"scales {exponents}, logits {logits}, kept {kept}")
    return got


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_at_the_ends_of_their_range(dim, code):
    bf16, code = torch.bfloat16, CODES[code]
    for kept in (0, 90):
        # tiny values: they and the outputs are bf16 numbers
        for e in (-105, -115, -120, -126):
            got = of_scales([e] * 8, [0, 1, 2, -3, 4, 0, 0, 1], dim, code, kept, bf16)
            assert (got[0] != 0).any()
            of_scales([e, e + 3, -126, e + 1, e, -126, e + 4, e], [9, 1, 2, -3, 4, 0, 0, 1], dim, code, kept, bf16)
        # an improbable block of large values beside a probable one of small values, either of them first
        for far, large, small in ((80, 100, -20), (84, 119, -2), (60, 110, 20), (80, 60, -60), (72, 115, 100)):
            of_scales([large, small] * 4, [-far, 0] * 4, dim, code, kept, bf16)
            of_scales([small, large] * 4, [0, -far] * 4, dim, code, kept, bf16)
            of_scales([small] * 7 + [large], [0] * 7 + [-far], dim, code, kept, bf16)
            of_scales([large] + [small] * 7, [-far] + [0] * 7, dim, code, kept, bf16)
    # a block that some tokens do not see yet, with a scale far above theirs
    of_scales([-100] * 7 + [120], [0, 1, 2, -3, 4, 0, 0, 1], dim, code, 0, bf16, counts=[20])


def test_nothing_but_empty_blocks():
    """Blocks of zeros have the least scale, or none yet."""
    for e in (-126.0, -math.inf):
        for kept in (0, 40):
            n, page, dim = 64, 16, 64
            table, pages = pages_for([n], page, 1, 1)
            c, s = torch.zeros((pages, 1, page, dim), device="cuda").to(E4M3), torch.full((pages, 1), 2.0 ** e, device="cuda")
            q = torch.randn((1, 4, dim), device="cuda", generator=generator(1)).bfloat16()
            select = torch.arange(kept, device="cuda", dtype=torch.int32)[None] if kept else None
            out, lse = ibwd.cache_attention(q, c, c, s, s, table, torch.tensor([n], device="cuda", dtype=torch.int32), select=select)
            assert (out == 0).all() and torch.allclose(lse, torch.full_like(lse, math.log(kept or n)), rtol=0, atol=2.0 ** -19)


@pytest.mark.parametrize("page,length", [(256, (1 << 30) + 700), (64, (1 << 31) - 1), (16, (1 << 31) - 20), (256, (1 << 31) - 1)])
def test_positions_up_to_the_largest(page, length):
    """A sequence as long as positions are numbers, most of whose pages are none: the others count wherever they lie."""
    dim, group, width = 64, 3, ((1 << 31) - 1) // page
    held = min(length, width * page)
    places = [0, 1, (1 << 29) // page, (1 << 30) // page - 1, (1 << 30) // page, (held - 1) // page - 1, (held - 1) // page]
    table = torch.full((1, width), -1, device="cuda", dtype=torch.int32)
    for i, at in enumerate(places):
        table[0, at] = 6 - i
    kc, ks = filled(7, 1, page, dim, E4M3, 1)
    vc, vs = filled(7, 1, page, dim, E4M3, 2)
    q = torch.randn((2, group, dim), device="cuda", generator=generator(3)).bfloat16()
    dl, cu = torch.tensor([length], device="cuda", dtype=torch.int32), offsets([2])
    # the same pages side by side, with as many positions in the last one
    near, n = torch.arange(6, -1, -1, device="cuda", dtype=torch.int32)[None], 6 * page + held - places[-1] * page
    # (the tokens see all that is held where the length is beyond it)
    first = max(0, min(length - 1, held) - places[-1] * page) + 6 * page
    select = torch.tensor([p * page + 5 for p in places] + [held - 1, 7], device="cuda", dtype=torch.int32).expand(2, 9).contiguous()
    close = torch.tensor([i * page + 5 for i in range(7)] + [n - 1, 7], device="cuda", dtype=torch.int32).expand(2, 9).contiguous()
    for ids, ids_near in ((None, None), (select, close)):
        got = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, cu=cu, select=ids)
        for i, seen in enumerate((first, n)):
            one = lambda t: None if t is None else t[i:i + 1]
            check_attention([t[i:i + 1] for t in got], q[i:i + 1], kc, vc, ks, vs, near, [seen], None, one(ids_near), dim ** -0.5, page,
                            f"{length} positions, token {i}")


def test_offsets_that_fall():
    """They leave the results undefined, but nothing around them is written, and the call is no longer than others: of 32768
    times the tokens it would be about 40 ms."""
    batch, tokens, dim = 1 << 16, 1 << 12, 64
    kc, ks = filled(4, 1, 16, dim, E4M3, 1)
    table = torch.zeros((batch, 2), device="cuda", dtype=torch.int32)
    lens = torch.full((batch,), 30, device="cuda", dtype=torch.int32)
    cu = torch.zeros(batch + 1, device="cuda", dtype=torch.int32)
    cu[1::2] = tokens
    q = torch.randn((tokens, 1, dim), device="cuda", generator=generator(1)).bfloat16()
    wide = torch.full((tokens + 2, 1, dim), 7.0, device="cuda", dtype=torch.bfloat16)
    times = []
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        ibwd.cache_attention(q, kc, kc, ks, ks, table, lens, cu=cu, out=wide[1:-1])
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert (wide[0] == 7).all() and (wide[-1] == 7).all() and min(times) < 10.0, times


def test_rows_before_the_first_sequence():
    """A part of a batch's offsets with all of its packed tokens: the rows of the others stay as they were."""
    lens, cu, page, dim = [20, 30, 0], [3, 5, 8, 8], 16, 64
    table, pages = pages_for(lens, page, 0, 1)
    kc, ks = filled(pages, 1, page, dim, E4M3, 1)
    vc, vs = filled(pages, 1, page, dim, E4M3, 2)
    q = torch.randn((10, 4, dim), device="cuda", generator=generator(3)).bfloat16()
    dl, offs = (torch.tensor(t, device="cuda", dtype=torch.int32) for t in (lens, cu))
    for kept in (0, 1, 200):
        select = torch.randint(-1, 30, (10, kept), device="cuda", generator=generator(4), dtype=torch.int32) if kept else None
        out = torch.full_like(q, 7)
        got = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, cu=offs, select=select, out=out)
        check_attention(got, q, kc, vc, ks, vs, table, lens, cu, select, dim ** -0.5, page, f"kept {kept}")
        assert (out[:3] == 7).all() and (out[8:] == 7).all()
    before = [t.clone() for t in (kc.view(torch.uint8), ks)]
    k = torch.randn((10, 1, dim), device="cuda", generator=generator(5)).bfloat16()
    ibwd.cache_write(k, None, kc, None, ks, None, table, dl, cu=offs)
    a, b = kc.clone(), ks.clone()
    kc.view(torch.uint8).copy_(before[0])
    ks.copy_(before[1])
    ibwd.cache_write(k[3:8].contiguous(), None, kc, None, ks, None, table, dl, cu=offs - 3)
    assert torch.equal(a.view(torch.uint8), kc.view(torch.uint8)) and torch.equal(b, ks)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_negative_scales(dim, code):
    """A code stands for code * scale whatever the scale's sign: the same numbers as with both turned."""
    lens, page, code = [300, 17, 1], 16, CODES[code]
    table, pages = pages_for(lens, page, 1, 1)
    kc, ks = filled(pages, 2, page, dim, code, 1, spread=2)
    vc, vs = filled(pages, 2, page, dim, code, 2, spread=2)
    q = torch.randn((3, 8, dim), device="cuda", generator=generator(3)).bfloat16()
    dl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    turned = [torch.where(torch.rand((pages, 2), device="cuda", generator=generator(i)) < 0.5, -1.0, 1.0) for i in (4, 5)]
    for kept in (0, 40):
        select = torch.randint(-1, 300, (3, kept), device="cuda", generator=generator(6), dtype=torch.int32) if kept else None
        want = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, select=select)
        codes = [(c.float() * t[:, :, None, None]).to(code) for c, t in ((kc, turned[0]), (vc, turned[1]))]
        got = ibwd.cache_attention(q, *codes, ks * turned[0], vs * turned[1], table, dl, select=select)
        # (rounding is the same for both signs)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(ibwd.cache_read(codes[1], vs * turned[1], table, dl, 300), ibwd.cache_read(vc, vs, table, dl, 300))
