"""Layer norms and their gradients against plain definitions in 64 bits."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, DT, U32, close, half_step, ld, out, padding_untouched, randn, tiny

pytestmark = pytest.mark.gpu


def depth(n):
    """Additions one after the other on the way of any value of a row to its sum, at most: a wave's
    lanes share the row, then lanes and waves are joined."""
    return n / 64 + 24


def workspace(nbytes):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)


def norm(x, gamma, beta, eps, dtype, pad=0, inplace=False, keep=True):
    import dense_gemm_tile_amd as dgt
    M, N = x.shape
    y = x if inplace else out(M, N, dtype=dtype, pad=pad)
    mean, rstd = (out(1, M)[0], out(1, M)[0]) if keep else (None, None)
    dgt.gemm_norm(M, N, dtype, x, ld(x), gamma, beta, eps, y, ld(y), mean, rstd, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return y, mean, rstd


def check_forward(x, gamma, beta, eps, dtype, got):
    y, mean, rstd = got
    x = x.double()
    n = x.shape[1]
    D = depth(n)
    m = x.mean(1, keepdim=True)
    em = D * U32 * x.abs().mean(1, keepdim=True) + tiny("f32")
    diff = x - m
    v = (diff * diff).mean(1, keepdim=True)
    # each difference is off by the mean's error and one rounding; the first cancels but for its square
    ev = (D + 4) * U32 * v + em * em + 2 * em * U32 * diff.abs().mean(1, keepdim=True)
    r = (v + eps) ** -0.5
    rel = 0.5 * ev / (v + eps) + 4 * U32
    u = diff * r
    eu = (r * (em + U32 * diff.abs()) + u.abs() * rel) * (1 + rel) + 2 * U32 * u.abs()
    g = torch.ones(n, dtype=torch.float64, device=DEV) if gamma is None else gamma.double()
    b = torch.zeros(n, dtype=torch.float64, device=DEV) if beta is None else beta.double()
    want = u * g + b
    tol = eu * g.abs() + 2 * U32 * ((u * g).abs() + b.abs())
    close(y, want, tol * 1.01 + half_step(dtype) * want.abs() + tiny(dtype), "Y")
    if mean is not None:
        close(mean, m[:, 0], em[:, 0], "mean")
        close(rstd, r[:, 0], (r * rel * 1.1)[:, 0], "rstd")


def check_grad(dy, x, gamma, mean, rstd, r, dtype, dx, dgamma, dbeta):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    M, N = x.shape
    g = torch.ones(N, dtype=torch.float64, device=DEV) if gamma is None else gamma.double()
    u, h = (x - mean) * rstd, dy * g
    D = depth(N)
    s1, s2 = h.mean(1, keepdim=True), (h * u).mean(1, keepdim=True)
    e1, e2 = (D + 2) * U32 * h.abs().mean(1, keepdim=True), (D + 5) * U32 * (h * u).abs().mean(1, keepdim=True)
    want = rstd * (h - s1 - u * s2)
    tol = rstd * (e1 + u.abs() * e2 + 6 * U32 * (h.abs() + s1.abs() + (u * s2).abs()))
    if r is not None:
        want = want + r.double()
        tol = tol + U32 * want.abs()
    if dx is not None:
        close(dx, want, tol * 1.01 + half_step(dtype) * want.abs() + tiny(dtype), "dX")
    if dgamma is not None:
        close(dgamma, (dy * u).sum(0), (M + 6) * U32 * (dy * u).abs().sum(0) + tiny("f32"), "dgamma")
    if dbeta is not None:
        close(dbeta, dy.sum(0), (M + 6) * U32 * dy.abs().sum(0) + tiny("f32"), "dbeta")


def both(gen, M, N, dtype, pad=0, offset=0.0, gamma=True, beta=True, residual=False, inplace=False, eps=1e-5,
         want=("dx", "dgamma", "dbeta")):
    import dense_gemm_tile_amd as dgt
    say(f"norm {M}x{N} {dtype} pad={pad} offset={offset} {gamma} {beta} {residual} {inplace}")
    x = randn(gen, M, N, dtype=dtype, pad=pad)
    x += offset
    gm = randn(gen, 1, N, dtype=dtype)[0] if gamma else None
    bt = randn(gen, 1, N, dtype=dtype)[0] if beta else None
    kept = x.clone()
    got = norm(x, gm, bt, eps, dtype, pad, inplace)
    check_forward(kept, gm, bt, eps, dtype, got)
    assert padding_untouched(got[0])
    if inplace:
        x.copy_(kept)
    _, mean, rstd = got
    dy = randn(gen, M, N, dtype=dtype, pad=pad)
    r = randn(gen, M, N, dtype=dtype, pad=pad) if residual else None
    dy0, r0 = dy.clone(), None if r is None else r.clone()
    dx = (dy if inplace is True else r if inplace == "r" else out(M, N, dtype=dtype, pad=pad)) if "dx" in want else None
    dg = out(1, N)[0] if "dgamma" in want else None
    db = out(1, N)[0] if "dbeta" in want else None
    size = dgt.gemm_norm_grad_workspace(M, N)
    dgt.gemm_norm_grad(M, N, dtype, dy, ld(dy), x, ld(x), gm, mean, rstd, r, ld(r), dx, ld(dx), dg, db, workspace(size),
                       size, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    check_grad(dy0, kept, gm, mean, rstd, r0, dtype, dx, dg, db)
    if dx is not None:
        assert padding_untouched(dx)


SIZES = [(1, 1), (1, 8), (3, 7), (33, 64), (5, 513), (7, 1024), (6, 1500), (100, 2048), (9, 2056), (40, 4096),
         (5, 5000), (3, 8192), (4, 8200), (2, 16384), (3, 16391), (2, 40000), (1025, 72), (3000, 130)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N", SIZES)
def test_norm_and_its_gradient(dtype, M, N):
    need_gpu()
    gen = torch.Generator().manual_seed(M * 31 + N)
    both(gen, M, N, dtype)
    both(gen, M, N, dtype, pad=3, offset=4.0, residual=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_norm_without_parameters_and_in_place(dtype):
    need_gpu()
    gen = torch.Generator().manual_seed(5)
    for M, N in ((17, 96), (6, 4096), (5, 1031), (3, 33000)):
        both(gen, M, N, dtype, gamma=False, beta=False)
        both(gen, M, N, dtype, beta=False, inplace=True)
        both(gen, M, N, dtype, residual=True, inplace="r", pad=8)
        for want in (("dx",), ("dgamma",), ("dbeta",), ("dgamma", "dbeta")):
            both(gen, M, N, dtype, want=want)


def test_row_ends_and_starts():
    """Every number of columns past the last whole piece, at pitches that put rows at any address."""
    need_gpu()
    gen = torch.Generator().manual_seed(6)
    for i in range(16):
        for base in (0, 512, 4096):
            both(gen, 9, base + i + 1, ("f16", "bf16", "f32")[i % 3], pad=i % 5, residual=i % 2 == 0)


def test_constant_rows_and_large_numbers():
    """A row of one value has no variance: U is 0 and Y is beta. Its gradient has the size of 1 / sqrt(eps)."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    for N in (1, 64, 1000, 4096, 33000):
        say(f"constant rows of {N}")
        x = torch.full((3, N), 2.5, dtype=torch.float32, device=DEV)
        x[1] = -1e18
        x[2] = 0
        beta = torch.arange(N, dtype=torch.float32, device=DEV) / N
        y, mean, rstd = norm(x, None, beta, 1e-5, "f32")
        # the mean of equal numbers is off by a few half steps of them, which (x - mean) then holds
        assert torch.allclose(y[2], beta, rtol=0, atol=0)
        close(mean, x[:, 0].double(), depth(N) * U32 * x[:, 0].double().abs() + 1e-45, "mean")
        off = depth(N) * U32 * 2.5
        close(y[0:1], beta.double()[None], torch.full_like(y[0:1], off / 1e-5 ** 0.5, dtype=torch.float64) + 2 * U32, "Y")
        assert torch.isfinite(y).all() and torch.isfinite(rstd).all()


def test_nan_stays_in_its_row():
    need_gpu()
    for N in (72, 4096, 40000):
        x = torch.randn(5, N, generator=torch.Generator().manual_seed(1)).to(DEV, torch.bfloat16)
        clean, _, _ = norm(x.clone(), None, None, 1e-5, "bf16")
        x[2, N // 2] = float("nan")
        x[3, 0] = float("inf")
        y, mean, rstd = norm(x, None, None, 1e-5, "bf16")
        assert torch.isnan(y[2]).all() and torch.isnan(rstd[2]) and torch.isnan(y[3]).any()
        assert torch.equal(y[[0, 1, 4]], clean[[0, 1, 4]])


def test_gradient_is_the_slope():
    """Against differences of the definition, in 64 bits."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(7)
    M, N, eps, h = 3, 12, 1e-3, 1e-5
    x, dy, gamma = (torch.randn(M, N, generator=gen).to(DEV) for _ in range(3))
    gamma = gamma[0].contiguous()

    def f(x, g):
        m = x.mean(1, keepdim=True)
        return (dy.double() * ((x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps) * g)).sum()
    _, mean, rstd = norm(x, gamma, None, eps, "f32")
    dx, dg = out(M, N), out(1, N)[0]
    size = dgt.gemm_norm_grad_workspace(M, N)
    dgt.gemm_norm_grad(M, N, "f32", dy, N, x, N, gamma, mean, rstd, None, 0, dx, N, dg, None, workspace(size), size,
                       stream=torch.cuda.current_stream())
    x64, g64 = x.double(), gamma.double()
    for i in range(M):
        for j in range(N):
            e = torch.zeros_like(x64)
            e[i, j] = h
            d = (f(x64 + e, g64) - f(x64 - e, g64)) / (2 * h)
            # h^2 / 6 of a third derivative below 1e4 here, and float32 arithmetic
            assert abs(float(dx[i, j]) - float(d)) < 1e-5, (i, j)
    for j in range(N):
        e = torch.zeros_like(g64)
        e[j] = h
        assert abs(float(dg[j]) - float((f(x64, g64 + e) - f(x64, g64 - e)) / (2 * h))) < 1e-5


def test_no_rows_gives_zero_sums_and_runs_repeat():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    dg, db = out(1, 40)[0], out(1, 40)[0]
    size = dgt.gemm_norm_grad_workspace(0, 40)
    dgt.gemm_norm_grad(0, 40, "bf16", None, 40, None, 40, None, None, None, None, 0, None, 0, dg, db, workspace(size), size)
    torch.cuda.synchronize()
    assert torch.equal(dg, torch.zeros_like(dg)) and torch.equal(db, torch.zeros_like(db))
    gen = torch.Generator().manual_seed(8)
    x, dy = (randn(gen, 3000, 520, dtype="bf16") for _ in range(2))
    _, mean, rstd = norm(x, None, None, 1e-5, "bf16")
    first = None
    for _ in range(3):
        dx, dg, db = out(3000, 520, dtype="bf16"), out(1, 520)[0], out(1, 520)[0]
        size = dgt.gemm_norm_grad_workspace(3000, 520)
        dgt.gemm_norm_grad(3000, 520, "bf16", dy, 520, x, 520, None, mean, rstd, None, 0, dx, 520, dg, db, workspace(size),
                           size, stream=torch.cuda.current_stream())
        got = (dx, dg, db)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
