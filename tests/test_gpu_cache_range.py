"""The attention over the 8-bit cache at the ends of its range: large logits, scales of any value."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from test_gpu_cache import CODES, E4M3, filled, generator, pages_for
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
