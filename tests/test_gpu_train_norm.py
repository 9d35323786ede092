"""Layer norm, forward and backward, against plain 64-bit forms."""
import pytest
import torch

import sparse_attention_indexer_bwd_gb300 as ibwd
from train_ref import DTYPES, check_norm_bwd, check_norm_fwd, norm_fwd

pytestmark = pytest.mark.gpu

WIDTHS = [1, 2, 7, 8, 31, 32, 64, 100, 128, 129, 136, 255, 256, 512, 513, 1000, 1024, 2047, 2048, 4096, 4104, 5001,
          8192, 9000, 16384, 16385, 40000]


def matrix(rows, n, dtype, pad=0, offset=0, seed=0, shift=0.5):
    """[rows, n] normal values of row-dependent size and offset, in rows of n + pad, `offset` elements into a buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(rows * (n + pad) + offset, device="cuda", generator=g)
    x = buf[offset:].view(rows, n + pad)
    x *= torch.rand((rows, 1), device="cuda", generator=g) * 2 + 0.25
    x += shift * torch.randn((rows, 1), device="cuda", generator=g)
    return buf.to(dtype)[offset:].view(rows, n + pad)[:, :n]


def weights(n, dtype=torch.float32, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((1 + 0.2 * torch.randn(n, device="cuda", generator=g)).to(dtype),
            (0.3 * torch.randn(n, device="cuda", generator=g)).to(dtype))


def same(a, b):
    view = {4: torch.int32, 2: torch.int16}
    return torch.equal(a.contiguous().view(view[a.element_size()]), b.contiguous().view(view[b.element_size()]))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", WIDTHS)
def test_forward_and_backward_over_widths(n, kind):
    dt = DTYPES[kind]
    for rows in (1, 5, 333):
        x = matrix(rows, n, dt, seed=n + rows)
        gamma, beta = weights(n)
        y, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta, eps=1e-6)
        check_norm_fwd((y, mean, rstd), x, gamma, beta, 1e-6, dt, f"{rows}x{n}")
        dy = matrix(rows, n, dt, seed=n + rows + 1)
        got = ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma)
        check_norm_bwd(got, dy, x, mean, rstd, gamma, f"{rows}x{n}")


@pytest.mark.parametrize("rows,n", [(4099, 128), (3001, 96), (2500, 1024), (20011, 40), (700, 4096), (450, 6000),
                                    (1500, 4104), (1400, 8192), (1300, 12288), (900, 16384)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_many_rows(rows, n, kind):
    dt = DTYPES[kind]
    x, dy = matrix(rows, n, dt, seed=3), matrix(rows, n, dt, seed=4)
    gamma, beta = weights(n)
    y, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta)
    check_norm_fwd((y, mean, rstd), x, gamma, beta, 1e-5, dt, f"{rows}x{n}")
    check_norm_bwd(ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma), dy, x, mean, rstd, gamma, f"{rows}x{n}")


@pytest.mark.parametrize("n", [128, 250, 4096, 4100, 20000])
@pytest.mark.parametrize("types", [("bf16", "fp32", "bf16"), ("fp16", "fp32", "fp16"), ("fp32", "bf16", "bf16"),
                                   ("fp32", "fp16", "fp16"), ("fp32", "fp32", "fp32")])
def test_mixed_types_and_weights(n, types):
    xt, dyt, yt = (DTYPES[t] for t in types)
    x, dy = matrix(77, n, xt, seed=5), matrix(77, n, dyt, seed=6)
    for wt in {torch.float32, xt}:
        gamma, beta = weights(n, wt)
        for g, b in ((gamma, beta), (gamma, None), (None, beta), (None, None)):
            got = ibwd.layer_norm_fwd(x, g, b, out_dtype=yt)
            assert got[0].dtype == yt
            check_norm_fwd(got, x, g, b, 1e-5, yt, f"{types} {wt}")
            check_norm_bwd(ibwd.layer_norm_bwd(dy, x, got[1], got[2], g), dy, x, got[1], got[2], g, f"{types} {wt}")


@pytest.mark.parametrize("n,pad,offset", [(128, 8, 0), (128, 64, 8), (128, 3, 0), (127, 1, 1), (2047, 64, 0),
                                          (4096, 8, 8), (4096, 1, 0), (4095, 1, 0), (1000, 24, 3)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_strides_and_alignments(n, pad, offset, kind):
    dt = DTYPES[kind]
    x, dy = matrix(211, n, dt, pad, offset, seed=7), matrix(211, n, dt, pad + 8, 0, seed=8)
    gamma, beta = weights(n)
    y, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta)
    check_norm_fwd((y, mean, rstd), x, gamma, beta, 1e-5, dt, "strided")
    check_norm_bwd(ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma), dy, x, mean, rstd, gamma, "strided")
    # the same bits from contiguous copies of the same alignment class or not: within the bounds, and the
    # columns between the rows stay as they were
    buf = torch.full((211, n + 8), 7.0, device="cuda", dtype=dt)
    ibwd.layer_norm_fwd(x, gamma, beta, out=buf[:, :n])
    check_norm_fwd((buf[:, :n], None, None), x, gamma, beta, 1e-5, dt, "strided out")
    assert (buf[:, n:] == 7).all()
    buf.fill_(7)
    ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma, out=buf[:, :n])
    assert (buf[:, n:] == 7).all()
    # unaligned weights
    w = torch.cat([gamma[:1], gamma, beta])
    got = ibwd.layer_norm_fwd(x, w[1:n + 1], w[n + 1:])
    check_norm_fwd(got, x, gamma, beta, 1e-5, dt, "unaligned weights")


@pytest.mark.parametrize("rows,n,pad", [(1500, 333, 0), (1500, 333, 5), (2001, 1001, 0), (1203, 2051, 2), (1100, 4099, 0),
                                        (640, 7001, 3), (400, 9001, 0), (333, 16383, 1), (320, 12288, 0), (40, 20001, 0),
                                        (7, 2049, 0), (9, 2049, 0), (33, 650, 4)])
@pytest.mark.parametrize("kind,dy_kind", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_unaligned_rows(rows, n, pad, kind, dy_kind):
    """Rows that begin anywhere in a 16-byte block, alike in all matrices or not, several of them a team."""
    dt = DTYPES[kind]
    x, dy = matrix(rows, n, dt, pad, seed=21), matrix(rows, n, DTYPES[dy_kind], pad, seed=22)
    gamma, beta = weights(n)
    y, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta)
    check_norm_fwd((y, mean, rstd), x, gamma, beta, 1e-5, dt, f"{rows}x{n}+{pad}")
    got = ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma)
    check_norm_bwd(got, dy, x, mean, rstd, gamma, f"{rows}x{n}+{pad}")
    again = ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma)
    assert all(same(a, b) for a, b in zip(got, again))
    # another alignment of dy and dx
    dy2 = torch.cat([dy[:, :1], dy], 1)[:, 1:]
    out = torch.empty((rows, n + 3), device="cuda", dtype=dt)[:, :n]
    check_norm_bwd(ibwd.layer_norm_bwd(dy2, x, mean, rstd, gamma, out=out), dy, x, mean, rstd, gamma, "other alignment")


@pytest.mark.parametrize("n", [96, 128, 2047, 4096, 12000, 40000])
def test_in_place_and_reproducible(n):
    x, dy = matrix(301, n, torch.bfloat16, seed=9), matrix(301, n, torch.bfloat16, seed=10)
    gamma, beta = weights(n)
    y, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta)
    z = x.clone()
    ibwd.layer_norm_fwd(z, gamma, beta, out=z)
    assert same(z, y)
    got = ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma)
    for _ in range(3):
        assert all(same(a, b) for a, b in zip(got, ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma)))
    for which in (x, dy):
        other = {id(x): x.clone(), id(dy): dy.clone()}
        a = ibwd.layer_norm_bwd(other[id(dy)], other[id(x)], mean, rstd, gamma, out=other[id(which)])
        assert all(same(p, q) for p, q in zip(a, got))


def test_large_offset_keeps_the_variance():
    """Rows whose mean is 4000 times their deviation: the two-pass sum of squares keeps it."""
    for n in (128, 1000, 4096, 40000):
        x = matrix(9, n, torch.float32, seed=11, shift=0) + 4000
        got = ibwd.layer_norm_fwd(x)
        check_norm_fwd(got, x, None, None, 1e-5, torch.float32, f"offset {n}")
        assert (got[2].double() / norm_fwd(x, None, None, 1e-5)[2] - 1).abs().max() < 1e-3


def test_constant_rows_and_one_column():
    for n in (1, 128, 1000, 4096):
        x = torch.full((4, n), 3.25, device="cuda")
        y, mean, rstd = ibwd.layer_norm_fwd(x, None, None, eps=1e-4)
        assert (y == 0).all() and (mean == 3.25).all() and (rstd - 100).abs().max() < 1e-3
        dx, dg, db = ibwd.layer_norm_bwd(torch.ones_like(x), x, mean, rstd)
        assert dx.abs().max() <= 100 * 2.0 ** -20 and (dg == 0).all() and (db == 4).all()


def test_no_rows():
    x = torch.empty((0, 128), device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = ibwd.layer_norm_fwd(x)
    assert y.shape == (0, 128) and mean.shape == (0,)
    dx, dg, db = ibwd.layer_norm_bwd(x, x, mean, rstd)
    assert dx.shape == (0, 128) and (dg == 0).all() and (db == 0).all()


def test_nan_and_infinity_stay_in_their_rows():
    for n in (128, 333, 4096):
        x, dy = matrix(40, n, torch.bfloat16, seed=12), matrix(40, n, torch.bfloat16, seed=13)
        clean = ibwd.layer_norm_fwd(x)
        clean_dx = ibwd.layer_norm_bwd(dy, x, clean[1], clean[2])[0]
        z = x.clone()
        z[7, n // 2] = float("nan")
        z[8, 0] = float("inf")
        y, mean, rstd = ibwd.layer_norm_fwd(z)
        assert torch.isnan(y[7:9]).all()
        keep = [i for i in range(40) if i not in (7, 8)]
        assert same(y[keep], clean[0][keep])
        dx = ibwd.layer_norm_bwd(dy, z, mean, rstd)[0]
        assert torch.isnan(dx[7:9]).all() and same(dx[keep], clean_dx[keep])


def test_leading_dimensions_and_parts():
    x = matrix(6 * 35, 64, torch.bfloat16, seed=14).view(6, 35, 64)
    gamma, beta = weights(64)
    y, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta)
    assert y.shape == x.shape and mean.shape == (6, 35)
    check_norm_fwd((y, mean, rstd), x, gamma, beta, 1e-5, torch.bfloat16, "3 dims")
    assert ibwd.layer_norm_fwd(x, stats=False)[1:] == (None, None)
    dx, dg, db = ibwd.layer_norm_bwd(y, x, mean, rstd, gamma, weight_grads=False)
    assert dg is None and db is None
    assert same(dx, ibwd.layer_norm_bwd(y, x, mean, rstd, gamma)[0])


def test_gradient_against_differences():
    """The backward pass against central differences of the 64-bit forward pass."""
    for n in (5, 130):
        x, dy = matrix(3, n, torch.float32, seed=15), matrix(3, n, torch.float32, seed=16)
        gamma, beta = weights(n)
        _, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta, eps=1e-3)
        dx, dg, db = ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma)
        h = 1e-4

        def loss(x, gamma, beta):
            return (norm_fwd(x, gamma, beta, 1e-3)[0] * dy.double()).sum()

        for of, grad in ((0, dx), (1, dg), (2, db)):
            args = [x.double(), gamma.double(), beta.double()]
            flat = args[of].view(-1)
            for i in range(0, flat.numel(), 3):
                keep = flat[i].clone()
                flat[i] = keep + h
                up = loss(*args)
                flat[i] = keep - h
                down = loss(*args)
                flat[i] = keep
                # truncation h^2 f'''/6 and the kernel's fp32 sums
                assert abs((up - down) / (2 * h) - grad.view(-1)[i]) < 2e-5 * (1 + dy.abs().sum())


def test_other_stream_and_graph():
    x, dy = matrix(500, 1024, torch.bfloat16, seed=17), matrix(500, 1024, torch.bfloat16, seed=18)
    gamma, beta = weights(1024)
    y, mean, rstd = ibwd.layer_norm_fwd(x, gamma, beta)
    want = ibwd.layer_norm_bwd(dy, x, mean, rstd, gamma)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for how in (s, s.cuda_stream):
        y2, m2, r2 = ibwd.layer_norm_fwd(x, gamma, beta, stream=how)
        got = ibwd.layer_norm_bwd(dy, x, m2, r2, gamma, stream=how)
        s.synchronize()
        assert same(y2, y) and all(same(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y3, m3, r3 = ibwd.layer_norm_fwd(x, gamma, beta)
        got = ibwd.layer_norm_bwd(dy, x, m3, r3, gamma)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(y3, y) and all(same(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    """The last rows of a matrix of more than 2^31 elements."""
    rows, n = 8, 128
    step = (1 << 31) // 4 // 8 * 8 + 8
    buf = torch.empty(rows * step, device="cuda", dtype=torch.bfloat16)
    x = buf.as_strided((rows, n), (step, 1))
    x.copy_(matrix(rows, n, torch.bfloat16, seed=19))
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    y, mean, rstd = ibwd.layer_norm_fwd(x, out=y)
    check_norm_fwd((y, mean, rstd), x, None, None, 1e-5, torch.bfloat16, "far rows")
    dy = matrix(rows, n, torch.bfloat16, seed=20)
    got = ibwd.layer_norm_bwd(dy, x, mean, rstd, out=x.clone(memory_format=torch.contiguous_format))
    check_norm_bwd(got, dy, x.contiguous(), mean, rstd, None, "far rows")
