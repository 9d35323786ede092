"""The operators of an answering layer together, against plain torch; and what the training operators' tests hold of
calls in general: refusals, first use under capture, host threads, refused launches, other devices."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from heads_ref import angles, statistics, turn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def plain_heads(x, gamma, beta, norm, positions, freq):
    xh, _, _ = statistics(x, norm, 1e-6)
    z = xh * (1.0 if gamma is None else gamma.double()) + (0.0 if beta is None else beta.double())
    return turn(z, angles(positions, freq, None), 0, False).bfloat16()


def test_layer_against_plain_torch():
    """Prompts and three steps. Every stage is held to its own inputs: heads to their formula, caches to a step of the
    codes, scores and attention to the caches' values."""
    from serve_indexer import Layer
    prompts = [70, 1, 129]
    layer = Layer(3, 256)
    hist = [[], [], []]
    for step in range(4):
        counts = prompts if step == 0 else None
        n = sum(prompts) if step == 0 else 3
        h = torch.randn((n, 512), device="cuda", generator=torch.Generator(device="cuda").manual_seed(step)).bfloat16()
        q, iq, weight, cu = layer.step(h, counts)
        qkv = (h @ layer.w_qkv).unflatten(1, (-1, 128))
        at, pos = 0, []
        for b in range(3):
            m = prompts[b] if step == 0 else 1
            pos.append(torch.arange(int(layer.lens[b]) - m, int(layer.lens[b]), device="cuda"))
            at += m
        pos = torch.cat(pos)
        ref_q = plain_heads(qkv[:, :8], None, None, "rms", pos, layer.freq[0])
        ref_k = plain_heads(qkv[:, 8:10], None, None, "rms", pos, layer.freq[0])
        assert (q.float() - ref_q.float()).abs().max() <= 2.0 ** -7 * ref_q.float().abs().max()  # one rounding to bf16, and a neighbour's
        index = (h @ layer.w_index).unflatten(1, (-1, 64))
        ref_ik = plain_heads(index[:, -1:], layer.gamma[2], layer.beta, "layer", pos, layer.freq[1])
        for b in range(3):
            rows = slice(*(cu[b:b + 2].tolist())) if cu is not None else slice(b, b + 1)
            hist[b].append((ref_k[rows], qkv[rows, 10:], ref_ik[rows]))
        # the caches hold what was written: within half a step of e4m3 of the value, or of the block's smallest normal code,
        # twice over since a raised scale rounds again, and bf16's rounding of the keys
        for c, s, which in ((layer.k, layer.k_scale, 0), (layer.v, layer.v_scale, 1), (layer.index, layer.index_scale, 2)):
            back = ibwd.cache_read(c, s, layer.table, layer.lens, 256, dtype=torch.float32)
            for b in range(3):
                want = torch.cat([t[which] for t in hist[b]]).float()
                got = back[b, :len(want)]
                tol = (2.0 ** -4 + 2.0 ** -7) * want.abs() + 2.0 ** -9 * s.max() * 2
                assert ((got - want).abs() <= tol).all()
                assert (back[b, len(want):] == 0).all()
        if step == 0:
            continue
        chosen = layer.select(iq, weight, 32)
        keys = ibwd.cache_read(layer.index, layer.index_scale, layer.table, layer.lens, 256)[:, :, 0].float()
        scores = torch.einsum("bhs,bh->bs", torch.relu(torch.einsum("bhd,bsd->bhs", iq.float(), keys)), weight)
        kd = ibwd.cache_read(layer.k, layer.k_scale, layer.table, layer.lens, 256, dtype=torch.float32)
        vd = ibwd.cache_read(layer.v, layer.v_scale, layer.table, layer.lens, 256, dtype=torch.float32)
        out, lse = layer.attend(q, select=chosen)
        for b in range(3):
            n = int(layer.lens[b])
            ids = chosen[b][chosen[b] >= 0].long()
            assert len(ids) == min(32, n) and (ids < n).all() and len(set(ids.tolist())) == len(ids)
            # no position that was left out scores higher than a chosen one by more than the sums' rounding
            rest = torch.ones(n, dtype=torch.bool, device="cuda")
            rest[ids] = False
            if rest.any():
                size = (torch.relu(torch.einsum("hd,sd->hs", iq[b].float(), keys[b, :n])) * weight[b].abs()[:, None]).sum(0).max()
                assert scores[b, :n][rest].max() <= scores[b, ids].min() + 2.0 ** -16 * size
            for head in range(8):
                y = kd[b, ids, head // 4] @ q[b, head].float() * 128 ** -0.5
                p = torch.softmax(y, 0)
                ref = p @ vd[b, ids, head // 4]
                assert (out[b, head].float() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 2.0 ** -9 * (p @ vd[b, ids, head // 4].abs()).max()
                assert (lse[b, head] - torch.logsumexp(y, 0)).abs() <= 1e-4


def test_example_runs():
    import serve_indexer
    far = serve_indexer.main(steps=3, prompts=(90, 5, 33), length=128, kept=128)
    assert max(far) <= 2.0 ** -6  # everything is selected: two orders of the same sums


def heads_args(tokens=6, heads=4, dim=64, dtype=torch.bfloat16):
    q = torch.randn((tokens, heads, dim), device="cuda").to(dtype)
    return q, torch.arange(tokens, device="cuda"), torch.ones(dim // 2, device="cuda", dtype=torch.float64), torch.ones(dim, device="cuda")


def refused(status, call, *args, **kwargs):
    with pytest.raises(ibwd.IndexerBwdError) as e:
        call(*args, **kwargs)
    assert e.value.status == status


def test_refusals_of_heads():
    q, pos, f, w = heads_args()
    out = torch.full_like(q, 7)
    for bad in (q[..., ::2], q.long(), q.cpu(), q[0, 0], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            ibwd.qk_norm_rope_fwd(bad, None, pos, f, q_out=out)
    for k in (q[:-1], q[..., :32], q.half(), q.cpu()):
        with pytest.raises(ValueError):
            ibwd.qk_norm_rope_fwd(q, k, pos, f, q_out=out)
    for bad in (pos[:-1], pos.float(), pos.cpu(), pos[:, None], None):
        with pytest.raises(ValueError):
            ibwd.qk_norm_rope_fwd(q, None, bad, f, q_out=out)
    for bad in (f.half(), f[:, None], f.cpu(), None):
        with pytest.raises(ValueError):
            ibwd.qk_norm_rope_fwd(q, None, pos, bad, q_out=out)
    for bad in (w[:-1], w.half(), w.double(), w.cpu()):
        with pytest.raises(ValueError):
            ibwd.qk_norm_rope_fwd(q, None, pos, f, q_gamma=bad, q_out=out)
    for how in (dict(q_norm="batch"), dict(k_gamma=w), dict(start=-1), dict(axes=torch.zeros(32, device="cuda", dtype=torch.int32)),
                dict(q_gamma=w, q_beta=w.bfloat16(), q_norm="layer"), dict(k_out=q)):
        with pytest.raises(ValueError):
            ibwd.qk_norm_rope_fwd(q, None, pos, f, q_out=out, **how)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.qk_norm_rope_fwd, q, None, pos, f, start=2, q_out=out)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.qk_norm_rope_fwd, q, None, pos, f, q_norm="none", q_gamma=w, q_out=out)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.qk_norm_rope_fwd, q, None, pos, f, q_gamma=w, q_beta=w, q_out=out)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.qk_norm_rope_fwd, q, None, pos, f, eps=-1.0, q_out=out)
    with pytest.raises(ValueError):
        ibwd.qk_norm_rope_fwd(torch.randn((2, 1, 513), device="cuda"), None)
    # results that overlap themselves, and in place with other strides
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.qk_norm_rope_fwd, q, None, pos, f, q_out=out[:1].expand(6, 4, 64))
    wide = torch.zeros((6, 4, 80), device="cuda", dtype=torch.bfloat16)
    refused(ibwd.IBWD_ERR_INVALID_ARG, ibwd.qk_norm_rope_fwd, wide[..., :64], None, pos, f, q_out=wide.as_strided((6, 4, 64), (256, 64, 1)))
    for bad in (q[:-1], q.half(), q.double(), q[:, :3]):
        with pytest.raises((ValueError, ibwd.IndexerBwdError)):
            ibwd.qk_norm_rope_bwd(bad, None, q, None, pos, f, q_out=out)
    refused(ibwd.IBWD_ERR_WORKSPACE, ibwd.qk_norm_rope_bwd, q, None, q, None, pos, f, q_out=out, workspace=torch.empty(16, device="cuda"))
    refused(ibwd.IBWD_ERR_WORKSPACE, ibwd.qk_norm_rope_bwd, q, None, q, None, pos, f, q_out=out, workspace=torch.empty(1 << 20))
    with pytest.raises(ValueError):
        ibwd.qk_norm_rope_bwd(q, None, q, None, pos, f, q_out=out, workspace=torch.empty((1 << 10, 1 << 10), device="cuda").t())
    assert (out == 7).all()


def cache_args(dim=64, heads=2, page=16, code=torch.float8_e4m3fn):
    c = torch.zeros((4, heads, page, dim), device="cuda", dtype=torch.uint8).view(code)
    s = torch.full((4, heads), 5.0, device="cuda")
    table = torch.tensor([[0, 1], [2, 3]], device="cuda", dtype=torch.int32)
    return c, s, table, torch.tensor([17, 3], device="cuda", dtype=torch.int32)


def test_refusals_of_the_cache():
    c, s, table, lens = cache_args()
    k = torch.randn((2, 2, 64), device="cuda").bfloat16()
    v, vs = c.clone(), s.clone()
    good = (k, k, c, v, s, vs, table, lens)

    def write(**kw):
        names = ("k", "v", "k_cache", "v_cache", "k_scale", "v_scale", "page_table", "lens")
        return ibwd.cache_write(**{**dict(zip(names, good)), **kw})

    f8 = torch.float8_e4m3fn
    for bad in (dict(k=k.cpu()), dict(k=k[:, :1]), dict(k=k[..., :32]), dict(k=k.long()), dict(v=k.half()), dict(v=None), dict(v_cache=None),
                dict(v_scale=None), dict(k_cache=c.view(torch.uint8)), dict(k_cache=c.view(torch.int8)), dict(k_cache=c[:, :, ::2]), dict(k_cache=c[0]),
                dict(k_scale=s[:-1]), dict(k_scale=s.half()), dict(page_table=table.long()), dict(page_table=table[0]), dict(page_table=table.cpu()),
                dict(page_table=table.t()), dict(lens=lens.long()), dict(lens=lens[:-1]), dict(lens=lens.cpu()), dict(cu=lens), dict(cu=lens.long())):
        with pytest.raises(ValueError):
            write(**bad)
    refused(ibwd.IBWD_ERR_INVALID_ARG, write, k=k[:1], v=k[:1])          # one token a sequence
    refused(ibwd.IBWD_ERR_INVALID_ARG, write, v_cache=c, v_scale=vs)      # the same memory twice
    odd = torch.zeros((4, 2, 24, 64), device="cuda", dtype=torch.uint8).view(f8)
    refused(ibwd.IBWD_ERR_UNSUPPORTED, write, k_cache=odd, v_cache=odd.clone())
    thin = torch.zeros((4, 2, 16, 40), device="cuda", dtype=torch.uint8).view(f8)
    refused(ibwd.IBWD_ERR_UNSUPPORTED, write, k=k[..., :40], v=k[..., :40], k_cache=thin, v_cache=thin.clone())
    assert (s == 5).all() and (c.view(torch.uint8) == 0).all() and (v.view(torch.uint8) == 0).all()

    out = torch.full((2, 20, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    for bad in (dict(length=-1), dict(length=20, dtype=torch.float64), dict(length=21, out=out), dict(length=20, out=out.transpose(1, 2)),
                dict(length=20, out=out.cpu())):
        with pytest.raises(ValueError):
            ibwd.cache_read(c, s, table, lens, **bad)
    assert (out == 7).all()

    q = torch.randn((2, 4, 64), device="cuda").bfloat16()
    out = torch.full_like(q, 7)

    def attend(**kw):
        names = ("q", "k_cache", "v_cache", "k_scale", "v_scale", "page_table", "lens", "out")
        return ibwd.cache_attention(**{**dict(zip(names, (q, c, v, s, vs, table, lens, out))), **kw})

    for bad in (dict(q=q.cpu()), dict(q=q[:, :3], out=None), dict(q=q[..., :32], out=None), dict(out=out[:-1]), dict(out=out.half()), dict(out=out.transpose(0, 1)),
                dict(v_cache=v[:-1]), dict(v_cache=v.view(torch.int8)), dict(select=torch.zeros((2, 0), device="cuda", dtype=torch.int32)),
                dict(select=torch.zeros((1, 4), device="cuda", dtype=torch.int32)), dict(select=torch.zeros((2, 4), device="cuda")),
                dict(workspace=torch.zeros((1 << 12, 1 << 13), device="cuda").t())):
        with pytest.raises(ValueError):
            attend(**bad)
    refused(ibwd.IBWD_ERR_UNSUPPORTED, attend, q=q.float(), out=None)
    refused(ibwd.IBWD_ERR_INVALID_ARG, attend, scale=float("nan"))
    refused(ibwd.IBWD_ERR_INVALID_ARG, attend, q=q[:1], out=out[:1])
    refused(ibwd.IBWD_ERR_WORKSPACE, attend, workspace=torch.zeros(64, device="cuda"))
    refused(ibwd.IBWD_ERR_WORKSPACE, attend, workspace=torch.zeros(1 << 24))
    c2, s2, t2, l2 = cache_args(dim=80)
    refused(ibwd.IBWD_ERR_UNSUPPORTED, ibwd.cache_attention, torch.zeros((2, 4, 80), device="cuda").bfloat16(), c2, c2.clone(), s2, s2, t2, l2)
    assert (out == 7).all()
    assert ibwd.indexer_bwd_last_device_status() == ibwd.IBWD_OK


def test_other_devices_are_refused():
    from named_tensor import Named
    other = f"cuda:{torch.cuda.current_device() + 1}"
    q, c = Named((2, 4, 64), torch.bfloat16, other), Named((4, 2, 16, 64), torch.int8, other)
    s, t, n = Named((4, 2), torch.float32, other), Named((2, 2), torch.int32, other), Named((2,), torch.int32, other)
    for call in (lambda: ibwd.qk_norm_rope_fwd(q, None), lambda: ibwd.qk_norm_rope_bwd(q, None, q, None),
                 lambda: ibwd.cache_write(q, None, c, None, s, None, t, n), lambda: ibwd.cache_read(c, s, t, n, 4),
                 lambda: ibwd.cache_attention(q, c, c, s, s, t, n)):
        with pytest.raises(ValueError, match="current device"):
            call()


PROGRAM = """
import torch
import sparse_attention_indexer_bwd_gb300 as ibwd
q = torch.randn((2, 4, 64), device="cuda").bfloat16()
pos, f = torch.arange(2, device="cuda"), torch.ones(32, device="cuda")
c, v = (torch.zeros((4, 2, 16, 64), device="cuda", dtype=torch.int8) for _ in range(2))
s, vs = torch.zeros((4, 2), device="cuda"), torch.zeros((4, 2), device="cuda")
table = torch.tensor([[0, 1], [2, 3]], device="cuda", dtype=torch.int32)
lens = torch.ones(2, device="cuda", dtype=torch.int32)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, k = ibwd.qk_norm_rope_fwd(q, q[:, :2], pos, f)
    g = ibwd.qk_norm_rope_bwd(y, k, q, q[:, :2], pos, f)
    ibwd.cache_write(k, k, c, v, s, vs, table, lens)
    out, lse = ibwd.cache_attention(y, c, v, s, vs, table, lens)
    back = ibwd.cache_read(c, s, table, lens, 2)
graph.replay()
torch.cuda.synchronize()
assert (back[:, 0].float() - k.float()).abs().max() <= 0.02 and (back[:, 1] == 0).all()
assert torch.equal(out, back[:, 0].repeat_interleave(2, 1)) and all(torch.isfinite(t).all() for t in (g[0], g[1], g[2], g[4]))
print("captured")
"""


def test_first_call_inside_a_capture():
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


def test_threads():
    """Several host threads, a stream each, all operators at once."""
    q, pos, f, w = heads_args(200, 8, 128)
    c, s, table, _ = cache_args(128)
    lens = torch.tensor([30, 20], device="cuda", dtype=torch.int32)
    k = torch.randn((50, 2, 128), device="cuda").bfloat16()
    cu = torch.tensor([0, 30, 50], device="cuda", dtype=torch.int32)
    ibwd.cache_write(k, None, c, None, s, None, table, lens, cu=cu)

    def work():
        y = ibwd.qk_norm_rope_fwd(q, None, pos, f, q_gamma=w)[0]
        g = ibwd.qk_norm_rope_bwd(q, None, q, None, pos, f, q_gamma=w)
        mine, scale = torch.zeros_like(c.view(torch.uint8)).view(c.dtype), torch.zeros_like(s)
        ibwd.cache_write(k, None, mine, None, scale, None, table, lens, cu=cu)
        return [y, g[0], g[2], mine.view(torch.uint8), ibwd.cache_read(c, s, table, lens, 32), *ibwd.cache_attention(q[:50], c, c, s, s, table, lens, cu=cu)]

    want = work()
    torch.cuda.synchronize()
    bad = []

    def run():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = work()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(1)

    threads = [threading.Thread(target=run) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_a_refused_launch_is_not_the_next_calls_error():
    from test_gpu_train_errors import runtime
    rt = runtime()
    q, pos, f, w = heads_args()
    c, s, table, lens = cache_args()
    k = torch.randn((2, 2, 64), device="cuda").bfloat16()
    calls = [lambda: ibwd.qk_norm_rope_fwd(q, None, pos, f), lambda: ibwd.qk_norm_rope_bwd(q, None, q, None, pos, f),
             lambda: ibwd.cache_write(k, None, c, None, s, None, table, lens), lambda: ibwd.cache_read(c, s, table, lens, 8),
             lambda: ibwd.cache_attention(k, c, c, s, s, table, lens)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    for bad in calls:
        stream = torch.cuda.Stream()
        raw = ctypes.c_void_p(stream.cuda_stream)
        with torch.cuda.stream(stream):  # (its blocks are in the allocator before the capture)
            bad()
        stream.synchronize()
        assert rt.cudaStreamBeginCapture(raw, 2) == 0
        assert rt.cudaStreamSynchronize(raw) != 0  # not allowed there: the capture is over
        with torch.cuda.stream(stream):
            refused(ibwd.IBWD_ERR_CUDA, bad)
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(raw, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
        for good in calls:
            good()
        torch.cuda.synchronize()


def test_captures_with_other_work_between():
    """Copies, another library's kernels and a second stream between the calls of a captured step."""
    q, pos, f, w = heads_args(2, 4, 64)
    c, s, table, _ = cache_args()
    lens = torch.ones(2, device="cuda", dtype=torch.int32)
    src, dst = torch.randn_like(q), torch.empty_like(q)
    state = c.view(torch.uint8).clone(), s.clone()

    def step(stream):
        dst.copy_(src)
        y, k = ibwd.qk_norm_rope_fwd(dst, dst[:, :2], pos, f, q_gamma=w)
        y = y * 2
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ibwd.cache_write(k, None, c, None, s, None, table, lens)
        z = torch.zeros_like(y)
        z.add_(y)
        torch.cuda.current_stream().wait_stream(side)
        out, lse = ibwd.cache_attention(z, c, c, s, s, table, lens)
        back = ibwd.cache_read(c, s, table, lens, 3)
        g = ibwd.qk_norm_rope_bwd(out, k, dst, dst[:, :2], pos, f, q_gamma=w)
        back = back + 1
        return y, out, lse, back, g[0], g[2], g[4]

    want = [t.clone() for t in step(None)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(None)
    for _ in range(3):
        c.view(torch.uint8).copy_(state[0])
        s.copy_(state[1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_a_chain_that_reads_what_it_just_wrote():
    """Each call takes the one before's result, many times without a wait: nothing may begin before it is there."""
    q, pos, f, _ = heads_args(300, 32, 128)
    want = q
    for _ in range(30):
        want, _ = ibwd.qk_norm_rope_fwd(want, None, pos, f, q_norm="none")
        torch.cuda.synchronize()
    for _ in range(5):
        got = q
        for _ in range(30):
            got, _ = ibwd.qk_norm_rope_fwd(got, None, pos, f, q_norm="none")
        assert torch.equal(got, want)
    c, s, table, _ = cache_args(128)
    lens = torch.zeros(2, device="cuda", dtype=torch.int32)
    k = torch.randn((2, 2, 128), device="cuda").bfloat16()

    def loop(wait):
        c.view(torch.uint8).zero_()
        s.zero_()
        lens.zero_()
        x, outs = k, []
        for i in range(25):
            lens.add_(1)
            ibwd.cache_write(x, None, c, None, s, None, table, lens)
            x, _ = ibwd.cache_attention(x, c, c, s, s, table, lens, scale=3.0)
            x = ibwd.cache_read(c, s, table, lens, 32)[:, i] + x
            outs.append(x)
            if wait:
                torch.cuda.synchronize()
        return torch.stack(outs)

    want = loop(True)
    for _ in range(5):
        assert torch.equal(loop(False), want)
