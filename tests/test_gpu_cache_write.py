"""The 8-bit cache's write where a call's pieces are unlike, and at the largest floats."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from test_gpu_cache import CODES, DT, generator, offsets, pages_for, same_cache
from heads_ref import write_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_one_prompt_among_single_tokens(code, kind):
    """One prompt of several pages among 63 sequences that bring a token each, in pages of all sizes: pieces from one token to
    more than a block of threads holds, in one call. Afterwards each brings a larger token, and the older codes move."""
    code = CODES[code]
    for page, dim, prompt in ((16, 64, 400), (64, 128, 400), (256, 128, 450), (256, 32, 1500), (128, 512, 60)):
        for where in (0, 40, 63):
            lens = [5 + (37 * b) % (2 * page) for b in range(64)]
            counts = [1] * 64
            lens[where], counts[where] = prompt + 7, prompt
            table, pages = pages_for([n + 1 for n in lens], page, 3, 1)
            cache = (torch.randn((pages, 2, page, dim), device="cuda", generator=generator(2)) * 40).clamp(-127, 127).to(code)
            scale = torch.full((pages, 2), 2.0 ** -9, device="cuda")
            held, unit = cache.cpu().double(), scale.cpu().double()
            for step in range(2):
                n = sum(counts)
                x = (torch.randn((n, 2, dim), device="cuda", generator=generator(3 + step)) * (0.3 if step == 0 else 4.0)).to(DT[kind])
                cu = offsets(counts)
                ibwd.cache_write(x, None, cache, None, scale, None, table, torch.tensor(lens, device="cuda", dtype=torch.int32), cu=cu)
                held, unit = write_ref(x.cpu(), held.float().to(code), unit, table.cpu(), lens, cu.tolist(), page)
                same_cache(cache, scale, held, unit, f"page {page}, prompt at {where}, step {step}")
                lens, counts = [m + 1 for m in lens], [1] * 64


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_values_that_no_scale_of_whole_numbers_holds(kind):
    """Above 127 * 2^120 the code is the largest; what is beside it in its block is rounded as ever."""
    top = 127 * 2.0 ** 120
    most = torch.finfo(DT[kind]).max
    x = torch.zeros((1, 1, 16), dtype=DT[kind])
    x[0, 0, :6] = torch.tensor([most, -most, 1.5 * top, top, 2.0 ** 125, -math.inf], dtype=torch.float64).to(DT[kind])
    table, lens = torch.zeros((1, 1), device="cuda", dtype=torch.int32), torch.ones(1, device="cuda", dtype=torch.int32)
    for code, want in ((torch.int8, [127, -127, 127, 127, 32, -127]), (torch.float8_e4m3fn, None)):
        cache, scale = torch.zeros((1, 1, 16, 16), device="cuda").to(code), torch.zeros((1, 1), device="cuda")
        ibwd.cache_write(x.cuda(), None, cache, None, scale, None, table, lens)
        assert scale.item() == 2.0 ** 120
        got = cache[0, 0, 0, :6].float().tolist()
        if want is not None:
            assert got == want
        else:  # (the largest fp32 and bf16 are nearly 256 * 2^120)
            assert got == [256, -256, 192, 128, 32, -448]
