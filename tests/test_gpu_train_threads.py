"""The training operators called from several host threads."""
import ctypes
import threading
import time

import torch
import pytest

import sparse_attention_indexer_bwd_gb300 as ibwd

pytestmark = pytest.mark.gpu


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def run(calls, count):
    """Every call `count` times in a thread of its own, on a stream of its own; the statuses that were not OK."""
    bad = []
    start = threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        raw = ctypes.c_void_p(stream.cuda_stream)
        start.wait()
        for _ in range(count):
            rc = call(raw)
            if rc:
                bad.append(rc)
                break
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return bad


def test_sizes_of_one_kernel_in_two_threads():
    """Calls that take the same kernel with different amounts of shared memory (ctypes lets threads run beside
    each other)."""
    lib = ibwd.load()
    keep = []

    def norm(n):
        x = torch.randn((4, n), device="cuda")
        y, s = torch.empty_like(x), torch.empty(4, device="cuda")
        keep.extend((x, y, s))
        return lambda st: lib.ibwd_layer_norm_fwd(ptr(x), 0, n, None, None, 0, ptr(y), 0, n, ptr(s), ptr(s), 4, n, 1e-5, st)

    def norm_bwd(n):
        x, dy = torch.randn((4, n), device="cuda"), torch.randn((4, n), device="cuda")
        dx, s = torch.empty_like(x), torch.ones(4, device="cuda")
        keep.extend((x, dy, dx, s))
        return lambda st: lib.ibwd_layer_norm_bwd(ptr(dy), 0, n, ptr(x), 0, n, None, 0, ptr(s), ptr(s), ptr(dx), n, None,
                                                  None, 4, n, None, 0, st)

    def distill(v, k, rows=80):
        x = torch.randn((rows, v), device="cuda").bfloat16()
        ids = torch.zeros((rows, k), device="cuda", dtype=torch.int32)
        teacher, loss, dx = torch.zeros((rows, k), device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
        keep.extend((x, ids, teacher, loss, dx))
        return lambda st: lib.ibwd_distill_grad(ptr(x), 1, v, ptr(ids), ptr(teacher), k, 1.0, None, 1.0, ptr(loss), ptr(dx),
                                                v, rows, v, st)

    for pair in ((norm(5000), norm(8000)), (norm(9000), norm(16000)), (norm_bwd(5000), norm_bwd(16000)),
                 (distill(21000, 8), distill(31000, 900)), (norm(9000), norm(16000), distill(21000, 8), distill(31000, 900))):
        assert run(pair, 3000) == []


def test_other_threads_run_while_the_launch_queue_is_full():
    """A call that waits for room in the launch queue does not hold the interpreter."""
    x = torch.randn((4, 128), device="cuda")
    ids = torch.zeros((4, 2), device="cuda", dtype=torch.int32)
    teacher = torch.zeros((4, 2), device="cuda")
    y, mean, rstd = ibwd.layer_norm_fwd(x)
    _, entropy, lse, _, _ = ibwd.token_logprobs_fwd(x, ids[:, 0].contiguous())
    calls = [lambda: ibwd.layer_norm_fwd(x, out=y), lambda: ibwd.layer_norm_bwd(x, x, mean, rstd, out=y, weight_grads=False),
             lambda: ibwd.token_logprobs_fwd(x, None), lambda: ibwd.token_logprobs_bwd(x, None, lse, entropy, None, lse, out=y),
             lambda: ibwd.distill_fwd(x, ids, teacher), lambda: ibwd.distill_bwd(x, ids, teacher, lse, lse, out=y),
             lambda: ibwd.distill_grad(x, ids, teacher, out=y)]
    for call in calls:
        call()
        torch.cuda.synchronize()
        stop, gaps = threading.Event(), []

        def tick():
            last = time.perf_counter()
            while not stop.is_set():
                time.sleep(0.001)
                now = time.perf_counter()
                gaps.append(now - last)
                last = now

        t = threading.Thread(target=tick)
        t.start()
        begin = time.perf_counter()
        torch.cuda._sleep(int(0.4 * 1.9e9))  # 0.4 s of GPU time, while more calls come than the queue holds
        longest = 0.0
        while time.perf_counter() - begin < 3.0 and longest < 0.1:
            at = time.perf_counter()
            call()
            longest = max(longest, time.perf_counter() - at)
        stop.set()
        t.join()
        torch.cuda.synchronize()
        assert longest >= 0.1, "the queue was never full"
        assert max(gaps) < 0.5 * longest
