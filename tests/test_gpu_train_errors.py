"""A call that the CUDA runtime refuses leaves nothing behind for the calls after it."""
import ctypes

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd

pytestmark = pytest.mark.gpu


def runtime():
    for line in open("/proc/self/maps"):
        if "libcudart.so" in line:
            return ctypes.CDLL(line.split()[-1])
    pytest.skip("torch's CUDA runtime is not a library of its own")


def test_a_refused_launch_is_not_the_next_calls_error():
    """Launches into a capture that was invalidated, then valid calls of every kind."""
    rt = runtime()
    x = torch.randn((4, 512), device="cuda")
    wide = torch.randn((2, 20000), device="cuda")
    ids, teacher = torch.zeros((4, 2), device="cuda", dtype=torch.int32), torch.zeros((4, 2), device="cuda")
    q, k = torch.randn((1, 8, 4, 64), device="cuda").bfloat16(), torch.randn((1, 8, 64), device="cuda").bfloat16()
    w, idx = torch.randn((1, 8, 4), device="cuda"), torch.zeros((1, 8, 8), device="cuda", dtype=torch.int32)
    _, mean, rstd = ibwd.layer_norm_fwd(x)
    out, stats = torch.empty_like(x), torch.empty(4, device="cuda")
    lib = ibwd.load()

    def ptr(t):
        return ctypes.c_void_p(t.data_ptr())

    refused = [lambda st: lib.ibwd_layer_norm_fwd(ptr(x), 0, 512, None, None, 0, ptr(out), 0, 512, None, None, 4, 512, 1e-5, st),
               lambda st: lib.ibwd_token_logprobs_fwd(ptr(x), 0, 512, None, 1.0, None, ptr(stats), ptr(stats), None, None, 0,
                                                      4, 512, st),
               lambda st: lib.ibwd_distill_grad(ptr(x), 0, 512, ptr(ids), ptr(teacher), 2, 1.0, None, 1.0, ptr(stats),
                                                ptr(out), 512, 4, 512, st)]
    valid = [lambda: ibwd.layer_norm_fwd(x), lambda: ibwd.layer_norm_fwd(wide), lambda: ibwd.layer_norm_bwd(x, x, mean, rstd),
             lambda: ibwd.distill_grad(x, ids, teacher), lambda: ibwd.indexer_fwd(q, k, w, idx)]
    for call in valid:
        call()
    torch.cuda.synchronize()
    for bad in refused:
        for good in valid:
            stream = torch.cuda.Stream()
            raw = ctypes.c_void_p(stream.cuda_stream)
            assert rt.cudaStreamBeginCapture(raw, 2) == 0
            assert rt.cudaStreamSynchronize(raw) != 0  # not allowed there: the capture is over
            assert bad(raw) == ibwd.IBWD_ERR_CUDA
            graph = ctypes.c_void_p()
            assert rt.cudaStreamEndCapture(raw, ctypes.byref(graph)) != 0
            rt.cudaGetLastError()  # (of this copy of the runtime; the library has its own)
            good()
            torch.cuda.synchronize()
