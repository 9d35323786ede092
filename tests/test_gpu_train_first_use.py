"""The first call of a process, made while a stream is captured."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import sparse_attention_indexer_bwd_gb300 as ibwd
x = torch.randn((8, 512), device="cuda")
ids = torch.zeros((8, 2), device="cuda", dtype=torch.int32)
teacher = torch.zeros((8, 2), device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, mean, rstd = ibwd.layer_norm_fwd(x)
    dx, dg, db = ibwd.layer_norm_bwd(y, x, mean, rstd)
    logprob, entropy, lse, top, _ = ibwd.token_logprobs_fwd(x, ids[:, 0].contiguous(), top_n=3)
    loss, dl = ibwd.distill_grad(x, ids, teacher)
graph.replay()
torch.cuda.synchronize()
assert (y.mean(1).abs() < 1e-5).all() and (dg > 0).all()
assert (lse - torch.logsumexp(x, 1)).abs().max() < 1e-5 and torch.equal(top[:, 0].long(), x.argmax(1))
assert torch.isfinite(loss).all() and dl.sum(1).abs().max() < 1e-5
print("captured")
"""


def test_first_call_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]
