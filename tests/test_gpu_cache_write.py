"""The 8-bit cache's write at the largest floats."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from test_gpu_cache import DT

pytestmark = pytest.mark.gpu


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
