"""Norm and rotation of queries and keys, forward and backward, against plain 64-bit forms."""
import math

import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from heads_ref import angles, check_bwd, check_fwd, statistics, turn
from train_ref import DTYPES, U

pytestmark = pytest.mark.gpu
EPS = 1e-6


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(tokens, heads, dim, dtype, seed, pad=0, at=0):
    """[tokens, heads, dim] in rows of heads * dim + pad, from element `at` of them on."""
    g = generator(seed)
    buf = torch.randn((tokens, heads * dim + pad), device="cuda", generator=g)
    buf *= torch.rand((tokens, 1), device="cuda", generator=g) * 2 + 0.25
    buf += 0.3 * torch.randn((tokens, 1), device="cuda", generator=g)
    return buf.to(dtype)[:, at:at + heads * dim].unflatten(1, (heads, dim))


def weights(dim, norm, dtype, seed):
    if norm == "none":
        return None, None
    g = generator(seed)
    gamma = (1 + 0.2 * torch.randn(dim, device="cuda", generator=g)).to(dtype)
    return gamma, (0.2 * torch.randn(dim, device="cuda", generator=g)).to(dtype) if norm == "layer" else None


def run(q, k, pos, freq, q_norm, k_norm, w_dtype=torch.float32, dy_dtypes=None, check=True, **how):
    """Forward and backward, checked."""
    dim = q.shape[-1]
    qg, qb = weights(dim, q_norm, w_dtype, 1)
    kg, kb = weights(dim, k_norm, w_dtype, 2) if k is not None else (None, None)
    angle = None if pos is None else angles(pos, freq, how.get("axes"))
    start, inter = how.get("start", 0), how.get("interleaved", False)
    yq, yk = ibwd.qk_norm_rope_fwd(q, k, pos, freq, q_norm=q_norm, k_norm=k_norm, q_gamma=qg, q_beta=qb, k_gamma=kg,
                                   k_beta=kb, eps=EPS, **how)
    assert yq.is_contiguous() and yq.dtype == q.dtype
    types = dy_dtypes or (q.dtype, q.dtype)
    dyq = make(*q.shape, types[0], 11)
    dyk = None if k is None else make(*k.shape, types[1], 12)
    out = ibwd.qk_norm_rope_bwd(dyq, dyk, q, k, pos, freq, q_norm=q_norm, k_norm=k_norm, q_gamma=qg, k_gamma=kg, eps=EPS, **how)
    what = f"{tuple(q.shape)} {q_norm} {k_norm} {how}"
    check_fwd(yq, q, q_norm, qg, qb, EPS, angle, start, inter, what + " q")
    check_bwd((out[0], out[2], out[3]), dyq, q, q_norm, qg, EPS, angle, start, inter, what + " q")
    if k is None:
        assert yk is None and out[1] is None and out[4] is None
    else:
        check_fwd(yk, k, k_norm, kg, kb, EPS, angle, start, inter, what + " k")
        check_bwd((out[1], out[4], out[5]), dyk, k, k_norm, kg, EPS, angle, start, inter, what + " k")
    return (yq, yk), out


def frequencies(pairs, dtype=torch.float64):
    return (10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / max(1, pairs))).to(dtype)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dim", [1, 2, 5, 8, 16, 24, 29, 32, 40, 64, 80, 96, 127, 128, 136, 192, 256, 264, 500, 512])
def test_widths(dim, kind):
    for tokens, heads, kv in ((1, 1, 1), (7, 3, 2), (45, 16, 1)):
        q, k = make(tokens, heads, dim, DTYPES[kind], dim), make(tokens, kv, dim, DTYPES[kind], dim + 1)
        pos = torch.randint(0, 100000, (tokens,), device="cuda", generator=generator(3))
        for pairs, start in {(dim // 2, 0), (dim // 4, 0), (dim // 4, dim - 2 * (dim // 4)), (0, 0)}:
            for inter in (False, True):
                run(q, k, pos, frequencies(pairs), "rms", "layer", start=start, interleaved=inter)


@pytest.mark.parametrize("norms", [("rms", "rms"), ("layer", "layer"), ("none", "layer"), ("rms", "none"), ("none", "none")])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norms_weights_and_gradient_types(norms, kind):
    dt = DTYPES[kind]
    for dim in (64, 100, 128):
        q, k = make(33, 8, dim, dt, 1), make(33, 2, dim, dt, 2)
        pos = torch.arange(33, device="cuda", dtype=torch.int32)
        for w in {torch.float32, dt}:
            for types in ((dt, dt), (torch.float32, torch.float32), (dt, torch.float32)):
                run(q, k, pos, frequencies(dim // 4, torch.float32), *norms, w_dtype=w, dy_dtypes=types)
        run(q, None, pos, frequencies(dim // 2), norms[0], "rms")
        run(q, k, None, None, *norms)


@pytest.mark.parametrize("tokens,heads,kv,dim", [(4099, 32, 8, 128), (3001, 64, 1, 128), (20011, 1, 0, 64), (5000, 3, 5, 80),
                                                 (2003, 7, 2, 29), (700, 130, 4, 256), (611, 1, 1, 512), (9001, 33, 0, 32)])
def test_many_rows(tokens, heads, kv, dim):
    q = make(tokens, heads, dim, torch.bfloat16, 1)
    k = make(tokens, kv, dim, torch.bfloat16, 2) if kv else None
    pos = torch.randint(0, 1 << 20, (tokens,), device="cuda", generator=generator(4))
    run(q, k, pos, frequencies(dim // 2), "rms", "layer")


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_many_rows_of_whole_parts(dim, kind):
    """Enough rows for sixteen elements a lane, in every form that has them, and those next to them."""
    tokens = 1031
    for heads, kv in ((8, 1), (3, 5)):
        q, k = make(tokens, heads, dim, DTYPES[kind], 1, 8, 8), make(tokens, kv, dim, DTYPES[kind], 2)
        pos = torch.randint(0, 1 << 20, (tokens,), device="cuda", generator=generator(4))
        run(q, k, None, None, "rms", "rms")
        for pairs in {dim // 2, dim // 4, 8, dim // 4 * 2 - 4, 1}:
            for start in {0, 8, 2, dim - 2 * pairs}:
                if 2 * pairs + start <= dim:
                    for inter in (False, True):
                        run(q, k, pos, frequencies(pairs), *(("rms", "layer") if heads == 8 else ("layer", "none")), start=start,
                            interleaved=inter)
                        types = (DTYPES[kind], torch.float32) if start else (torch.float32, torch.float32)
                        run(q, k, pos, frequencies(pairs), *(("rms", "rms") if heads == 8 else ("none", "rms")), start=start,
                            interleaved=inter, dy_dtypes=None if inter else types)


@pytest.mark.parametrize("pad,at", [(256, 0), (256, 128), (8, 8), (3, 1), (1, 0)])
def test_heads_within_a_wider_buffer(pad, at):
    for dim in (64, 128, 20):
        q, k = make(21, 4, dim, torch.bfloat16, 5, pad, at), make(21, 2, dim, torch.bfloat16, 6, pad, at)
        pos = torch.arange(21, device="cuda") * 1000
        run(q, k, pos, frequencies(dim // 2), "rms", "rms")
        # heads in front of tokens
        qt = torch.randn((4, 21, dim), device="cuda", generator=generator(7)).bfloat16().transpose(0, 1)
        run(qt, k, pos, frequencies(dim // 2), "layer", "rms")


def test_axes():
    t, dim = 50, 96
    q, k = make(t, 6, dim, torch.float16, 1), make(t, 2, dim, torch.float16, 2)
    pos = torch.randint(0, 4000, (3, t), device="cuda", generator=generator(9))
    for axes in (torch.arange(48) * 3 // 48, torch.arange(48) % 3, torch.tensor([0, 5, -1, 2] * 12), torch.full((48,), 2)):
        axes = axes.to("cuda", torch.int32)
        for inter in (False, True):
            run(q, k, pos, frequencies(48), "rms", "rms", axes=axes, interleaved=inter)
            run(q, k, pos.int(), frequencies(48), "rms", "rms", axes=axes, interleaved=inter)
    # batches: [axes, batch, tokens]
    qb = q.unflatten(0, (5, 10))
    axes = (torch.arange(48, device="cuda") * 3 // 48).int()
    a, _ = ibwd.qk_norm_rope_fwd(q, None, pos, frequencies(48), axes=axes)
    b, _ = ibwd.qk_norm_rope_fwd(qb, None, pos.unflatten(1, (5, 10)), frequencies(48), axes=axes)
    assert torch.equal(a, b.flatten(0, 1))


def test_far_and_negative_positions():
    q = make(9, 2, 128, torch.float32, 3)
    pos = torch.tensor([0, 1, -1, -70000, 10**6, 2**31 - 1, -2**31, 123456789, 2**30], device="cuda")
    run(q, None, pos, frequencies(64), "rms", "rms")
    run(q, None, pos.int(), frequencies(64), "none", "rms")
    # frequencies of more than a turn, and negative ones
    run(q, None, pos[:5].repeat(2)[:9], -7.25 * frequencies(64), "none", "rms")


def test_in_place_and_reproducible():
    for dim in (128, 29):
        q, k = make(300, 8, dim, torch.bfloat16, 1), make(300, 2, dim, torch.bfloat16, 2)
        pos, f = torch.arange(300, device="cuda"), frequencies(dim // 2)
        a = ibwd.qk_norm_rope_fwd(q, k, pos, f)
        q2, k2 = q.clone(), k.clone()
        versions = q2._version, k2._version
        b = ibwd.qk_norm_rope_fwd(q2, k2, pos, f, q_out=q2, k_out=k2)
        assert b[0].data_ptr() == q2.data_ptr() and q2._version > versions[0] and k2._version > versions[1]
        assert torch.equal(a[0], q2) and torch.equal(a[1], k2)
        dq, dk = make(300, 8, dim, torch.bfloat16, 3), make(300, 2, dim, torch.bfloat16, 4)
        a = ibwd.qk_norm_rope_bwd(dq, dk, q, k, pos, f, "layer", "layer")
        b = ibwd.qk_norm_rope_bwd(dq, dk, q, k, pos, f, "layer", "layer")
        c = ibwd.qk_norm_rope_bwd(dq.clone(), dk, q.clone(), k, pos, f, "layer", "layer", q_out=dq.clone())
        for x, y, z in zip(a, b, c):
            assert torch.equal(x, y) and torch.equal(x, z)
        x, d = q.clone(), dq.clone()
        assert torch.equal(ibwd.qk_norm_rope_bwd(d, None, x, None, pos, f, "layer", q_out=x)[0], a[0])
        x, d = q.clone(), dq.clone()
        assert torch.equal(ibwd.qk_norm_rope_bwd(d, None, x, None, pos, f, "layer", q_out=d)[0], a[0])
        none = ibwd.qk_norm_rope_bwd(dq, dk, q, k, pos, f, "layer", "layer", weight_grads=False)
        assert torch.equal(none[0], a[0]) and none[2:] == (None,) * 4


def test_shared_gradients():
    """A gradient that all tokens or heads share, with steps of 0."""
    q = make(40, 6, 64, torch.bfloat16, 1)
    one = make(1, 6, 64, torch.bfloat16, 2)
    pos, f = torch.arange(40, device="cuda"), frequencies(32)
    for dy in (one.expand(40, 6, 64), make(40, 1, 64, torch.bfloat16, 3).expand(40, 6, 64)):
        a = ibwd.qk_norm_rope_bwd(dy, None, q, None, pos, f)
        b = ibwd.qk_norm_rope_bwd(dy.contiguous(), None, q, None, pos, f)
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_no_tokens():
    q = torch.empty((0, 4, 64), device="cuda")
    pos, f = torch.empty(0, device="cuda", dtype=torch.int64), frequencies(32)
    y, _ = ibwd.qk_norm_rope_fwd(q, None, pos, f)
    assert y.shape == q.shape
    out = ibwd.qk_norm_rope_bwd(q, None, q, None, pos, f, "layer")
    assert (out[2] == 0).all() and (out[3] == 0).all() and out[0].shape == q.shape


def test_nan_and_infinity_stay_in_their_heads():
    for dim in (128, 30):
        q = make(20, 4, dim, torch.float32, 1)
        pos, f = torch.arange(20, device="cuda"), frequencies(dim // 4)
        clean, _ = ibwd.qk_norm_rope_fwd(q, None, pos, f)
        bad = q.clone()
        bad[3, 1, 5] = math.nan
        bad[7, 2, 0] = math.inf
        y, _ = ibwd.qk_norm_rope_fwd(bad, None, pos, f)
        mask = torch.ones((20, 4), dtype=torch.bool, device="cuda")
        mask[3, 1] = mask[7, 2] = False
        assert torch.equal(y[mask], clean[mask])
        assert torch.isnan(y[3, 1]).all() and torch.isnan(y[7, 2]).any()
        # without a norm they stay in their pair
        y, _ = ibwd.qk_norm_rope_fwd(bad, None, pos, f, "none")
        p = dim // 4
        assert torch.isnan(y[3, 1]).sum() == 2 and torch.isnan(y[3, 1, [5, 5 + p]]).all()
        last = q.clone()
        last[3, 1, dim - 1] = math.inf  # not turned
        y, _ = ibwd.qk_norm_rope_fwd(last, None, pos, f, "none")
        assert y[3, 1, dim - 1] == math.inf and torch.isfinite(y[3, 1, :dim - 1]).all()


def test_zero_rows_and_extreme_sizes():
    q = torch.zeros((3, 2, 64), device="cuda", dtype=torch.bfloat16)
    q[1] = 2.0 ** 60
    q[2] = 2.0 ** -60
    pos, f = torch.zeros(3, device="cuda", dtype=torch.int32), frequencies(32)
    run(q, None, pos, f, "rms", "rms")
    assert (ibwd.qk_norm_rope_fwd(q, None, pos, f)[0][0] == 0).all()


def test_gradient_against_differences():
    """Central differences of sum(y dy) in fp32, along directions. Of a sum of n products the values' roundings leave
    noise = 64 u sum |y dy| in each of the two, the third derivative 50 h^2 |v|^3 r^3 sum |dy| (r the largest
    1 / standard deviation, 50 over the third derivatives of x / |x|)."""
    for dim, norm, inter in ((64, "layer", False), (48, "rms", True), (128, "none", False), (29, "layer", False)):
        q = torch.randn((6, 2, dim), device="cuda", generator=generator(1))
        dy = torch.randn((6, 2, dim), device="cuda", generator=generator(2))
        gamma, beta = weights(dim, norm, torch.float32, 3)
        pos, f = torch.arange(6, device="cuda") * 37, frequencies(dim // 4)
        how = dict(q_norm=norm, q_gamma=gamma, eps=EPS, interleaved=inter)
        dx, _, dgamma, dbeta, _, _ = ibwd.qk_norm_rope_bwd(dy, None, q, None, pos, f, **how)

        def value(x, g=gamma, b=beta):
            y, _ = ibwd.qk_norm_rope_fwd(x, None, pos, f, **{**how, "q_gamma": g}, q_beta=b)
            return (y.double() * dy.double()).sum().item(), (y.double() * dy.double()).abs().sum().item()

        _, r, _ = statistics(q, norm, EPS)
        for seed in range(3):
            v = torch.randn(q.shape, device="cuda", generator=generator(10 + seed))
            h = 2.0 ** -7
            plus, size = value(q + h * v)
            minus, _ = value(q - h * v)
            got = (dx.double() * v.double()).sum().item()
            # |v| of a head over sqrt(dim), in units of the head's size
            rel = (v.double().square().mean(-1).sqrt() * r[..., 0]).max().item()
            tol = 64 * U * size / h + 50 * (h * rel) ** 2 * rel * dy.double().abs().sum().item() * (norm != "none")
            tol += 64 * U * (dx.double() * v.double()).abs().sum().item() + 4 * U * q.abs().max().item() / h * dx.double().abs().sum().item()
            assert abs((plus - minus) / (2 * h) - got) <= tol, (dim, norm, (plus - minus) / (2 * h), got, tol)
        for w, grad, name in ((gamma, dgamma, "g"), (beta, dbeta, "b")):
            if w is None:
                continue
            v = torch.randn(dim, device="cuda", generator=generator(20))
            plus, size = value(q, **{name: w + v})
            minus, _ = value(q, **{name: w - v})
            got = (grad.double() * v.double()).sum().item()
            assert abs((plus - minus) / 2 - got) <= 128 * U * (size + (grad.double() * v.double()).abs().sum().item()) * 8


def test_other_stream_and_graph():
    q, k = make(100, 8, 128, torch.bfloat16, 1), make(100, 2, 128, torch.bfloat16, 2)
    pos, f = torch.arange(100, device="cuda"), frequencies(64)
    want = ibwd.qk_norm_rope_fwd(q, k, pos, f) + ibwd.qk_norm_rope_bwd(q, k, q, k, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ibwd.qk_norm_rope_fwd(q, k, pos, f, stream=side) + ibwd.qk_norm_rope_bwd(q, k, q, k, pos, f, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert (a is None and b is None) or torch.equal(a, b)
    static = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ibwd.qk_norm_rope_fwd(static, k, pos, f)
        g = ibwd.qk_norm_rope_bwd(static, k, static, k, pos, f)
    for seed in (5, 6):
        new = make(100, 8, 128, torch.bfloat16, seed)
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = ibwd.qk_norm_rope_fwd(new, k, pos, f)
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
        want = ibwd.qk_norm_rope_bwd(new, k, new, k, pos, f)
        assert torch.equal(g[0], want[0]) and torch.equal(g[2], want[2])


def test_offsets_past_32_bits():
    n = (1 << 31) // 1024 + 3
    buf = torch.empty((n, 1024), device="cuda", dtype=torch.bfloat16)
    q = buf[:, :128].view(n, 2, 64)
    rows = torch.tensor([0, 5, n - 3, n - 1], device="cuda")
    buf.zero_()
    q[rows] = make(4, 2, 64, torch.bfloat16, 1)
    pos = torch.arange(n, device="cuda")
    y, _ = ibwd.qk_norm_rope_fwd(q, None, pos, frequencies(32))
    check_fwd(y[rows], q[rows], "rms", None, None, 1e-6, angles(pos[rows], frequencies(32), None), 0, False, "far rows")
