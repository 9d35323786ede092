"""The 8-bit cache: written and read back, bit for bit, and the attention over it against a plain 64-bit form."""
import math
import random

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from heads_ref import check_attention, read_ref, scale_for, write_ref

pytestmark = pytest.mark.gpu

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
CODES = {"e4m3": E4M3, "int8": INT8}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def pages_for(lens, page, extra, seed, width=None):
    """A page table with the sequences' pages in random places, -1 behind them; (table, pages)."""
    counts = [-(-max(n, 0) // page) for n in lens]
    total = sum(counts) + extra
    order = list(range(total))
    random.Random(seed).shuffle(order)
    width = max(counts + [1]) if width is None else width
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    return table.cuda(), total


def filled(pages, heads, page, dim, code, seed, spread=0):
    """Random codes and power-of-two scales, `spread` the range of their exponents."""
    g = generator(seed)
    x = torch.randn((pages, heads, page, dim), device="cuda", generator=g)
    codes = (x * 30).round().clamp(-127, 127).to(INT8) if code == INT8 else (x * 100).clamp(-448, 448).to(E4M3)
    e = torch.randint(-spread, spread + 1, (pages, heads), device="cuda", generator=g) if spread else torch.zeros((pages, heads), device="cuda")
    return codes, torch.exp2(e.float() - (5 if code == INT8 else 6.0))


def offsets(counts):
    return torch.tensor([0] + [sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32, device="cuda")


def same_cache(codes, scale, held, unit, what):
    got = codes.cpu()
    a, b = got.double(), held
    assert torch.equal(torch.isnan(a), torch.isnan(b)), what
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)), what
    u = scale.cpu().double()
    assert torch.equal(torch.isnan(u), torch.isnan(unit)) and torch.equal(torch.nan_to_num(u), torch.nan_to_num(unit)), what


# -------------------------------------------------------------- write, read ---

@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page,dim,heads", [(16, 16, 1), (16, 64, 3), (32, 80, 2), (64, 128, 1), (128, 48, 2), (256, 32, 1), (16, 512, 1)])
def test_write_over_steps(page, dim, heads, code):
    """Prompts, then tokens one by one and by threes, then longer pieces; the older tokens' scales rise on the way."""
    code, kinds = CODES[code], ["bf16", "fp16", "fp32"]
    lens = [0, 0, 0]
    table, pages = pages_for([3 * page + 9, 2 * page, page + 1], page, 2, 1)
    ck, cv = (torch.zeros((pages, heads, page, dim), device="cuda").to(code) for _ in range(2))
    sk, sv = torch.zeros((pages, heads), device="cuda"), torch.zeros((pages, heads), device="cuda")
    refs = [(ck.cpu().double(), sk.cpu().double()), (cv.cpu().double(), sv.cpu().double())]
    steps = [[page + 3, 5, 0], [1, 1, 1], [3, 0, 2], [1, 2, 1], [page + 2, page - 9, 0]]
    for i, counts in enumerate(steps):
        dt = DT[kinds[i % 3]]
        lens = [n + c for n, c in zip(lens, counts)]
        n = sum(counts)
        k = (torch.randn((n, heads, dim), device="cuda", generator=generator(i)) * 3.0 ** i).to(dt)
        v = (torch.randn((n, heads, dim), device="cuda", generator=generator(50 + i)) * 0.01).to(dt)
        cu = None if counts == [1, 1, 1] else offsets(counts)
        ibwd.cache_write(k, v, ck, cv, sk, sv, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=cu)
        for which, (x, c, s) in enumerate(((k, ck, sk), (v, cv, sv))):
            held, unit = refs[which]
            h2, u2 = write_ref(x.cpu(), _as(held, code), unit, table.cpu(), lens, None if cu is None else cu.tolist(), page)
            refs[which] = (h2, u2)
            same_cache(c, s, h2, u2, f"step {i}")


def _as(held, code):
    return held.to(torch.float32).to(code)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_scales_at_the_edges(code):
    """Largest values at, just under and just over what a scale holds, the smallest and largest floats."""
    dt, code = torch.float32, CODES[code]
    top = 448.0 if code == E4M3 else 127.0
    edge = torch.tensor([top, top * 2 ** -20, top * 2 ** 30])
    values = torch.cat([edge, torch.nextafter(edge, torch.zeros(1)), torch.nextafter(edge, torch.full((1,), math.inf)),
                        torch.tensor([0.0, 2.0 ** -149, 1e-40, 1e-30, 3.4e38, torch.finfo(dt).max, 2.0 ** -126])])
    n = len(values)
    x = torch.randn((n, 1, 16), generator=torch.Generator().manual_seed(1)).clamp(-1, 1) * values[:, None, None] * 0.999
    x[:, 0, 3] = -values
    table, pages = pages_for([1] * n, 16, 1, 2)
    codes, scale = torch.zeros((pages, 1, 16, 16), device="cuda").to(code), torch.full((pages, 1), 7.0, device="cuda")
    held, unit = write_ref(x, codes.cpu(), scale.cpu(), table.cpu(), [1] * n, None, 16)
    ibwd.cache_write(x.cuda(), None, codes, None, scale, None, table, torch.ones(n, dtype=torch.int32, device="cuda"))
    same_cache(codes, scale, held, unit, "edges")
    got = scale[table[:, 0].long(), 0].cpu().tolist()
    for v, u in zip(values.tolist(), got):
        assert u == scale_for(v, code) and (v <= top * u or u == 2.0 ** 120)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_what_is_not_finite(code):
    code = CODES[code]
    x = torch.randn((4, 2, 32), device="cuda", generator=generator(1))
    x[0, 0, 4], x[1, 0, 5], x[2, 1, 6] = math.inf, -math.inf, math.nan
    table, pages = pages_for([40], 16, 1, 3)
    codes, scale = torch.zeros((pages, 2, 16, 32), device="cuda").to(code), torch.ones((pages, 2), device="cuda")
    for step in range(2):
        lens, cu = [20 + 4 * step], [0, 4]
        held, unit = write_ref(x.cpu(), codes.cpu(), scale.cpu(), table.cpu(), lens, cu, 16)
        ibwd.cache_write(x, None, codes, None, scale, None, table, torch.tensor(lens, device="cuda", dtype=torch.int32),
                         cu=torch.tensor(cu, device="cuda", dtype=torch.int32))
        same_cache(codes, scale, held, unit, f"step {step}")
    y = ibwd.cache_read(codes, scale, table, torch.tensor([24], device="cuda", dtype=torch.int32), 24, dtype=torch.float32)
    assert torch.isnan(y[0, 18, 1]).any() and torch.isfinite(y[0, 16:, 0]).all()


def test_pages_lengths_and_offsets_that_are_none():
    """Nothing outside is written, read or attended to: pages out of range, lengths beyond the table or below 0, offsets
    beyond the tokens."""
    page, heads, dim = 16, 2, 64
    table = torch.tensor([[0, 9, 2], [-1, 4, 5], [6, 7, -7], [8, 1 << 30, 3]], dtype=torch.int32, device="cuda")
    codes, scale = filled(9, heads, page, dim, E4M3, 1)
    for lens, counts, tokens in (([40, 33, 48, 20], [3, 33, 20, 1], 57), ([-5, 100, 3, 47], [4, 70, 9, 2], 85),
                                 ([40, 33, 48, 20], [3, 33, 20, 50], 70)):
        cu = offsets(counts)
        x = torch.randn((tokens, heads, dim), device="cuda", generator=generator(2)).bfloat16()
        c, s = codes.clone(), scale.clone()
        cut = [min(v, tokens) for v in cu.tolist()]
        held, unit = write_ref(x.cpu(), c.cpu(), s.cpu(), table.cpu(), lens, cut, page)
        dl = torch.tensor(lens, device="cuda", dtype=torch.int32)
        ibwd.cache_write(x, None, c, None, s, None, table, dl, cu=cu)
        same_cache(c, s, held, unit, str(lens))
        y = ibwd.cache_read(c, s, table, dl, 60, dtype=torch.float32)
        assert torch.equal(y.double(), read_ref(c, s, table, lens, 60, page))
        q = torch.randn((tokens, 4, dim), device="cuda", generator=generator(3)).bfloat16()
        out = ibwd.cache_attention(q, c, c, s, s, table, dl, cu=cu)
        check_attention(out, q, c, c, s, s, table, lens, cut, None, dim ** -0.5, page, str(lens))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page,heads,dim", [(16, 1, 16), (64, 1, 128), (32, 5, 80), (256, 2, 512), (128, 8, 64)])
def test_read(page, heads, dim, code, kind):
    code = CODES[code]
    lens = [0, 1, page - 1, page, 3 * page + 5]
    table, pages = pages_for(lens, page, 2, 4)
    codes, scale = filled(pages, heads, page, dim, code, 5, spread=8)
    dl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    for length in (1, page, 2 * page + 3, 4 * page + 1):
        y = ibwd.cache_read(codes, scale, table, dl, length, dtype=DT[kind])
        ref = read_ref(codes, scale, table, lens, length, page)
        assert torch.equal(y, ref.to(DT[kind]))
        out = torch.full_like(y, 7)
        version = out._version
        assert ibwd.cache_read(codes, scale, table, dl, length, out=out) is not None and torch.equal(out, y)
        assert out._version > version
    assert ibwd.cache_read(codes, scale, table, dl, 0).shape == (5, 0, heads, dim)


def test_heads_in_a_wider_buffer_and_versions():
    page, heads, dim = 32, 4, 64
    lens = [45, 32]
    table, pages = pages_for(lens, page, 1, 6)
    dl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    wide = torch.randn((77, 3 * heads * dim + 5), device="cuda", generator=generator(1)).bfloat16()
    for at in (0, heads * dim, 3):
        k, v = (wide[:, o:o + heads * dim].unflatten(1, (heads, dim)) for o in (at, at + heads * dim))
        got = []
        for a, b in ((k, v), (k.contiguous(), v.contiguous())):
            c = [torch.zeros((pages, heads, page, dim), device="cuda").to(E4M3) for _ in range(2)]
            s = [torch.zeros((pages, heads), device="cuda") for _ in range(2)]
            versions = [t._version for t in c + s]
            ibwd.cache_write(a, b, *c, *s, table, dl, cu=offsets(lens))
            assert all(t._version > w for t, w in zip(c + s, versions))
            got.append([t.view(torch.uint8) for t in c] + s)
        assert all(torch.equal(a, b) for a, b in zip(*got))


# ---------------------------------------------------------------- attention ---

def attend(lens, counts, heads, group, dim, page, code, kind="bf16", kept=0, seed=0, spread=0, scale=None, duplicate=False):
    table, pages = pages_for(lens, page, 2, seed)
    kc, ks = filled(pages, heads, page, dim, code, seed + 1, spread)
    vc, vs = filled(pages, heads, page, dim, code, seed + 2, spread)
    n = len(lens) if counts is None else sum(counts)
    cu = None if counts is None else offsets(counts)
    q = (1.5 * torch.randn((n, heads * group, dim), device="cuda", generator=generator(seed + 3))).to(DT[kind])
    select = None
    if kept:
        select = torch.randint(-2, max(lens) + 3, (n, kept), device="cuda", generator=generator(seed + 4), dtype=torch.int32)
        if not duplicate:  # distinct ones
            select = torch.stack([torch.randperm(max(lens) + 5, device="cuda", generator=generator(seed + 5 + i))[:kept] - 2
                                  if max(lens) + 5 >= kept else
                                  torch.cat([torch.randperm(max(lens) + 5, device="cuda")[:kept] - 2,
                                             torch.full((kept - max(lens) - 5,), -1, device="cuda")]) for i in range(n)]).int()
    dl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    got = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, cu=cu, select=select, scale=scale)
    check_attention(got, q, kc, vc, ks, vs, table, lens, None if cu is None else cu.tolist(), select,
                    dim ** -0.5 if scale is None else scale, page, f"{lens} {counts} {heads}x{group}x{dim} page {page} kept {kept}")
    return got


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(page, dim, code):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 130, 0, 1000, 257]
    for heads, group in ((1, 1), (2, 4), (3, 7), (1, 16), (2, 17), (1, 64)):
        attend(lens, None, heads, group, dim, page, CODES[code], seed=dim + heads)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_several_tokens(dim, code):
    for counts, lens in (([3, 0, 1, 5], [100, 7, 64, 5]), ([4, 4], [4, 300]), ([1, 2, 70], [3, 1, 90]), ([5], [3])):
        for heads, group in ((1, 1), (2, 4), (2, 6), (1, 12)):
            attend(lens, counts, heads, group, dim, 32, CODES[code], "fp16", seed=len(lens))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_selected(dim, code):
    for kept in (1, 15, 64, 100, 333):
        for heads, group in ((1, 16), (2, 5), (1, 33)):
            attend([300, 40, 1, 129], None, heads, group, dim, 16, CODES[code], kept=kept, seed=kept)
            attend([300, 40, 9], [3, 5, 2], heads, group, dim, 64, CODES[code], kept=kept, seed=kept + 1)
    attend([50, 70], None, 2, 4, dim, 16, CODES[code], kept=90, duplicate=True)


@pytest.mark.parametrize("heads,group,lens", [(1, 8, [70000]), (2, 4, [30000, 1, 20001]), (1, 1, [131072]), (4, 16, [9000, 8000])])
def test_long(heads, group, lens):
    for dim in (64, 128, 256):
        attend(lens, None, heads, group, dim, 64, E4M3, seed=7)


def test_large_and_ragged_batches():
    rng = random.Random(5)
    lens = [rng.choice([0, 1, 5, 17, 64, 200, 333, 700]) for _ in range(300)]
    attend(lens, None, 2, 4, 128, 16, E4M3, seed=1)
    counts = [min(n, rng.choice([0, 1, 2, 5])) for n in lens]
    attend(lens, counts, 1, 3, 64, 32, INT8, seed=2)
    attend(lens[:40], counts[:40], 2, 3, 64, 32, INT8, kept=77, seed=3)


@pytest.mark.parametrize("dim,group", [(128, 16), (64, 16), (128, 30), (256, 9), (64, 41)])
def test_many_rows_whose_items_end_in_neighbouring_blocks(dim, group):
    """Items of two to four tiles, so that nearly every block ends one that another began."""
    rng = random.Random(dim + group)
    lens = [rng.choice([129, 200, 300, 390, 500]) for _ in range(330)]
    attend(lens, None, 1, group, dim, 32, E4M3, seed=4)
    attend(lens[:170], [rng.choice([1, 2, 3]) for _ in range(170)], 2, group, dim, 16, INT8, seed=5)
    attend(lens, None, 1, group, dim, 16, INT8, kept=300, seed=6)
    # and of many parts each
    attend([9000, 12345, 1, 7000], None, 1, group, dim, 64, E4M3, seed=8)


def test_scales_far_apart():
    """Blocks whose scales differ by up to 2^24, and by 2^200."""
    for dim in (64, 128):
        attend([500, 77], None, 2, 4, dim, 16, E4M3, seed=1, spread=6, scale=0.001)
        attend([500, 77], None, 1, 4, dim, 16, INT8, seed=1, spread=12, scale=1e-6)
    lens, page, dim = [48], 16, 64
    table, pages = pages_for(lens, page, 0, 1)
    kc, ks = filled(pages, 1, page, dim, E4M3, 1)
    vc, vs = filled(pages, 1, page, dim, E4M3, 2)
    vs[table[0, 1]] = 2.0 ** 100
    vs[table[0, 2]] = 2.0 ** -100
    q = torch.randn((1, 4, dim), device="cuda", generator=generator(3)).bfloat16()
    dl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    got = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl)
    check_attention(got, q, kc, vc, ks, vs, table, lens, None, None, dim ** -0.5, page, "far apart")
    vs[:] = 0  # nothing but zeros
    out, lse = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl)
    assert (out == 0).all() and torch.equal(lse, got[1])


@pytest.mark.parametrize("size", [2.0 ** -100, 1e-20, 1e4, 1e30])
def test_queries_of_any_size(size):
    """Tiny and huge queries, with a scale that brings the logits back."""
    lens, page, dim = [200], 16, 128
    table, pages = pages_for(lens, page, 0, 1)
    kc, ks = filled(pages, 1, page, dim, E4M3, 1)
    vc, vs = filled(pages, 1, page, dim, E4M3, 2)
    q = (torch.randn((1, 4, dim), device="cuda", generator=generator(3)) * size).bfloat16()
    got = ibwd.cache_attention(q, kc, vc, ks, vs, table, torch.tensor(lens, device="cuda", dtype=torch.int32), scale=0.1 / size)
    check_attention(got, q, kc, vc, ks, vs, table, lens, None, None, 0.1 / size, page, str(size))


def test_peaked_and_flat_logits():
    for scale in (0.0, 1e-4, 3.0, -1.0):
        attend([700, 65], None, 2, 4, 128, 64, E4M3, scale=scale)


@pytest.mark.parametrize("dim,heads,group", [(64, 2, 4), (64, 1, 8), (128, 2, 3), (128, 1, 8), (256, 1, 4), (256, 2, 8)])
def test_invisible_nan(dim, heads, group):
    """NaN keys and values that some tokens see and others do not, and behind a sequence's end."""
    page = 16
    lens, counts = [30, 40], [4, 1]
    table, pages = pages_for([48, 48], page, 1, 1)
    kc, ks = filled(pages, heads, page, dim, E4M3, 1)
    vc, vs = filled(pages, heads, page, dim, E4M3, 2)
    q = torch.randn((5, heads * group, dim), device="cuda", generator=generator(3)).bfloat16()
    dl, cu = torch.tensor(lens, device="cuda", dtype=torch.int32), offsets(counts)
    clean = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, cu=cu)
    check_attention(clean, q, kc, vc, ks, vs, table, lens, [0, 4, 5], None, dim ** -0.5, page, "clean")

    def poison(c, b, at, dims=slice(None)):
        c.view(torch.uint8)[table[b, at // page].long(), :, at % page, dims] = 0x7F

    kn, vn = kc.clone(), vc.clone()
    for c in (kn, vn):  # behind the ends
        poison(c, 0, 30)
        poison(c, 0, 47)
        poison(c, 1, 40)
    got = ibwd.cache_attention(q, kn, vn, ks, vs, table, dl, cu=cu)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    # position 28 is seen by the first sequence's tokens 2 and 3 alone
    for c in (kn, vn):
        poison(c, 0, 28, slice(5, 6))
    for k, v in ((kn, vc), (kc, vn), (kn, vn)):
        got = ibwd.cache_attention(q, k, v, ks, vs, table, dl, cu=cu)
        for t in (0, 1, 4):
            assert torch.isfinite(got[0][t].float()).all()
            assert (got[0][t].float() - clean[0][t].float()).abs().max() <= 2.0 ** -7 * clean[0][t].float().abs().max()
            assert torch.equal(got[1][t], clean[1][t])
        for t in (2, 3):
            if k is kn:
                assert torch.isnan(got[1][t]).all() and torch.isnan(got[0][t]).all()
            else:
                assert torch.isnan(got[0][t, :, 5]).all() and torch.equal(got[1][t], clean[1][t])
                assert torch.isfinite(got[0][t, :, 6:].float()).all()
    # not selected
    select = torch.tensor([[27, 3], [3, 2], [1, 27], [3, 27], [39, 1]], device="cuda", dtype=torch.int32)
    got = ibwd.cache_attention(q, kn, vn, ks, vs, table, dl, cu=cu, select=select)
    assert torch.isfinite(got[0].float()).all()
    # a NaN query is its own token's
    bad = q.clone()
    bad[1, 2, 3] = math.nan
    got = ibwd.cache_attention(bad, kc, vc, ks, vs, table, dl, cu=cu)
    assert torch.isnan(got[0][1, 2]).all() and torch.isnan(got[1][1, 2])
    keep = torch.ones((5, heads * group), dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][keep], clean[1][keep])


def test_nan_scales_of_whole_numbers():
    """A block of int8 values whose scale is NaN is NaN for those that see it, and for nobody else."""
    page, dim = 16, 64
    table, pages = pages_for([48, 48], page, 0, 1)
    kc, ks = filled(pages, 1, page, dim, INT8, 1)
    vc, vs = filled(pages, 1, page, dim, INT8, 2)
    q = torch.randn((4, 4, dim), device="cuda", generator=generator(3)).bfloat16()
    dl, cu = torch.tensor([34, 40], device="cuda", dtype=torch.int32), offsets([3, 1])
    clean = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, cu=cu)
    for which in range(2):
        scales = [ks.clone(), vs.clone()]
        scales[which][table[0, 2].long()] = math.nan  # positions 32 on: tokens 1 and 2 of the first sequence see them
        got = ibwd.cache_attention(q, kc, vc, *scales, table, dl, cu=cu)
        for t in (0, 3):
            assert (got[0][t].float() - clean[0][t].float()).abs().max() <= 2.0 ** -7 * clean[0][t].float().abs().max()
            assert (got[1][t] - clean[1][t]).abs().max() <= 1e-5
        for t in (1, 2):
            assert torch.isnan(got[0][t]).all()
            assert torch.isnan(got[1][t]).all() if which == 0 else torch.equal(got[1][t], clean[1][t])


def test_rows_behind_the_last_sequence():
    table, pages = pages_for([20, 30], 16, 0, 1)
    kc, ks = filled(pages, 1, 16, 64, E4M3, 1)
    q = torch.randn((9, 4, 64), device="cuda", generator=generator(3)).bfloat16()
    dl = torch.tensor([20, 30], device="cuda", dtype=torch.int32)
    for select in (None, torch.zeros((9, 2), device="cuda", dtype=torch.int32)):
        out = torch.full_like(q, 7)
        ibwd.cache_attention(q, kc, kc, ks, ks, table, dl, cu=offsets([2, 3]), select=select, out=out)
        assert (out[5:] == 7).all() and (out[:5] != 7).any(-1).all()


def test_strided_queries_leading_dimensions_and_workspace():
    table, pages = pages_for([200, 300], 16, 0, 1)
    kc, ks = filled(pages, 2, 16, 128, E4M3, 1)
    vc, vs = filled(pages, 2, 16, 128, E4M3, 2)
    dl = torch.tensor([200, 300], device="cuda", dtype=torch.int32)
    wide = torch.randn((2, 8 * 128 + 13), device="cuda", generator=generator(3)).bfloat16()
    for at in (0, 8, 13, 1):
        q = wide[:, at:at + 1024 if at + 1024 <= wide.shape[1] else None][:, :1024].unflatten(1, (8, 128))
        a = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl)
        work = torch.empty(ibwd.cache_attention_workspace_size(128), device="cuda", dtype=torch.uint8)
        b = ibwd.cache_attention(q.contiguous()[:, None], kc, vc, ks, vs, table, dl, workspace=work, out=torch.empty((2, 1, 8, 128), device="cuda", dtype=q.dtype))
        assert torch.equal(a[0], b[0][:, 0]) and torch.equal(a[1], b[1][:, 0])


def test_streams_graphs_and_repeats():
    table, pages = pages_for([400, 90, 1000], 16, 4, 1, width=70)
    kc, ks = filled(pages, 2, 16, 128, E4M3, 1)
    vc, vs = filled(pages, 2, 16, 128, E4M3, 2)
    q = torch.randn((3, 8, 128), device="cuda", generator=generator(3)).bfloat16()
    dl = torch.tensor([400, 90, 1000], device="cuda", dtype=torch.int32)
    want = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl)
    for _ in range(5):
        got = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ibwd.cache_attention(q, kc, vc, ks, vs, table, dl, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    # a decoding step as a graph: a token is written, read back and attended to, lengths and values changing between replays
    k1, v1 = torch.randn((3, 2, 128), device="cuda").bfloat16(), torch.randn((3, 2, 128), device="cuda").bfloat16()
    lens = dl.clone()
    args = (kc, vc, ks, vs)
    graph = torch.cuda.CUDAGraph()
    state = [t.clone() for t in args]
    with torch.cuda.graph(graph):
        ibwd.cache_write(k1, v1, *args, table, lens)
        out = ibwd.cache_attention(q, *args, table, lens)
        back = ibwd.cache_read(kc, ks, table, lens, 1100)
    for n in (0, -30, -60):
        for t, s in zip(args, state):
            t.copy_(s)
        lens.copy_(dl + n)
        k1.normal_(generator=generator(10 - n))
        graph.replay()
        torch.cuda.synchronize()
        mine = [s.clone() for s in state]
        ibwd.cache_write(k1, v1, *mine, table, lens)
        ref = ibwd.cache_attention(q, *mine, table, lens)
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
        assert torch.equal(back, ibwd.cache_read(mine[0], mine[2], table, lens, 1100))


def test_offsets_past_32_bits():
    page, heads, dim = 256, 8, 256
    pages = (1 << 32) // (page * heads * dim) + 5
    kc = torch.zeros((pages, heads, page, dim), device="cuda", dtype=torch.uint8).view(E4M3)
    ks = torch.ones((pages, heads), device="cuda")
    table = torch.tensor([[pages - 1, 2, pages - 3]], device="cuda", dtype=torch.int32)
    lens = torch.tensor([600], device="cuda", dtype=torch.int32)
    k = torch.randn((600, heads, dim), device="cuda", generator=generator(1)).bfloat16()
    ibwd.cache_write(k, None, kc, None, ks, None, table, lens, cu=offsets([600]))
    sub = table[0].long()
    held, unit = write_ref(k.cpu(), torch.zeros((3, heads, page, dim)).to(E4M3), torch.ones((3, heads)), torch.tensor([[0, 1, 2]]), [600], [0, 600], page)
    same_cache(kc[sub], ks[sub], held, unit, "far pages")
    y = ibwd.cache_read(kc, ks, table, lens, 600, dtype=torch.float32)
    assert torch.equal(y.double(), read_ref(kc[sub], ks[sub], torch.tensor([[0, 1, 2]], device="cuda"), [600], 600, page))
    q = torch.randn((1, heads, dim), device="cuda", generator=generator(2)).bfloat16()
    got = ibwd.cache_attention(q, kc, kc, ks, ks, table, lens)
    check_attention(got, q, kc[sub], kc[sub], ks[sub], ks[sub], torch.tensor([[0, 1, 2]], device="cuda"), [600], None, None, dim ** -0.5, page, "far")
