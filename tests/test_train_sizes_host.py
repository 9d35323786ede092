"""Sizes beyond the C types are refused before they are cut to them."""
import ctypes

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from named_tensor import Named

WIDE = (1 << 32) + 128


def test_wide_rows():
    """2^32 + 128 columns are not 128."""
    x, r = Named((1, WIDE), torch.bfloat16), Named((1,))
    ids, t = Named((1, 2), torch.int32), Named((1, 2))
    for call in (lambda: ibwd.layer_norm_fwd(x), lambda: ibwd.layer_norm_bwd(x, x, r, r),
                 lambda: ibwd.token_logprobs_fwd(x), lambda: ibwd.token_logprobs_bwd(x, None, r, r, None, r),
                 lambda: ibwd.distill_fwd(x, ids, t), lambda: ibwd.distill_bwd(x, ids, t, r, r),
                 lambda: ibwd.distill_grad(x, ids, t)):
        with pytest.raises(ValueError, match="too wide"):
            call()
    assert ibwd.layer_norm_bwd_workspace_size(4, WIDE) == 0


@pytest.mark.parametrize("n,fits", [(1 << 30, False), ((1 << 30) - 20, False), ((1 << 30) - 64, True), (1 << 20, True)])
def test_widths_whose_column_sums_pass_an_int(n, fits):
    """Refused before the first kernel, which would write what the second one cannot be launched for."""
    lib = ibwd.load()
    p, out = ctypes.c_void_p(4096), ctypes.c_void_p(8192)  # never dereferenced

    def call(sums):
        return lib.ibwd_layer_norm_bwd(p, 0, n, p, 0, n, None, 0, p, p, out, n, sums, sums, 1, n, p, 0, None)

    assert (call(p) != ibwd.IBWD_ERR_UNSUPPORTED) == fits
    assert (ibwd.layer_norm_bwd_workspace_size(1, n) > 0) == fits
    assert call(None) != ibwd.IBWD_ERR_UNSUPPORTED  # without sums any width


@pytest.mark.gpu
def test_many_alternatives_and_slots():
    x = torch.zeros((1, 64), device="cuda")
    for n in (65, WIDE, 1 << 31, (1 << 31) + 5, -WIDE):
        with pytest.raises(ibwd.IndexerBwdError) as e:
            ibwd.token_logprobs_fwd(x, top_n=n)
        assert e.value.status == ibwd.IBWD_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="too many"):
        ibwd.distill_fwd(x, Named((1, WIDE), torch.int32), Named((1, WIDE)))
