"""Workspaces that do not lie in one piece are refused before anything is read or launched."""
import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd


def test_workspaces_with_gaps_or_repeats():
    x, r = torch.zeros((4, 64)), torch.zeros(4)
    whole = torch.zeros((64, 64))
    for bad in (whole.view(-1)[:1].expand(1 << 20), whole.view(-1)[::2], whole.t()):
        with pytest.raises(ValueError, match="workspace"):
            ibwd.layer_norm_bwd(x, x, r, r, workspace=bad)
        with pytest.raises(ValueError, match="x: expected a CUDA tensor"):
            ibwd.layer_norm_bwd(x, x, r, r, workspace=bad, weight_grads=False)  # takes none
    with pytest.raises(ValueError, match="x: expected a CUDA tensor"):
        ibwd.layer_norm_bwd(x, x, r, r, workspace=whole)
