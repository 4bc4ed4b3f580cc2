"""gemm_norm_grad with dX = X, and gemm_norm with Y = X: the same results as with matrices of their own."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, ld, out, padding_untouched, randn
from test_layer_norm_gpu import check_grad, norm, workspace

pytestmark = pytest.mark.gpu

# Rows that fill no workgroup (four, two and one of them at a time), the widest rows held in registers, and longer ones.
SIZES = [(1, 64), (5, 64), (6, 1000), (7, 1024), (2050, 130), (2049, 520), (3, 2048), (5, 2056), (6, 4096), (9, 8192), (3, 8200),
         (2, 16391)]


def grad(M, N, dtype, dy, x, gamma, mean, rstd, r, dx):
    import dense_gemm_tile_amd as dgt
    dg, db, size = out(1, N)[0], out(1, N)[0], dgt.gemm_norm_grad_workspace(M, N)
    dgt.gemm_norm_grad(M, N, dtype, dy, ld(dy), x, ld(x), gamma, mean, rstd, r, ld(r), dx, ld(dx), dg, db, workspace(size), size,
                       stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return dg, db


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N", SIZES)
def test_gradient_over_x(dtype, M, N):
    need_gpu()
    gen = torch.Generator().manual_seed(M + N)
    for pad, residual in ((0, True), (3, False)):
        say(f"norm_grad over X {M}x{N} {dtype} pad={pad}")
        x, dy = randn(gen, M, N, dtype=dtype, pad=pad), randn(gen, M, N, dtype=dtype, pad=pad)
        r = randn(gen, M, N, dtype=dtype, pad=pad) if residual else None
        gamma = randn(gen, 1, N, dtype=dtype)[0]
        _, mean, rstd = norm(x, gamma, None, 1e-5, dtype, pad)
        dx, kept = out(M, N, dtype=dtype, pad=pad), x.clone()
        sums = grad(M, N, dtype, dy, x, gamma, mean, rstd, r, dx)
        check_grad(dy, kept, gamma, mean, rstd, r, dtype, dx, *sums)
        over = grad(M, N, dtype, dy, x, gamma, mean, rstd, r, x)
        assert torch.equal(x, dx) and torch.equal(over[0], sums[0]) and torch.equal(over[1], sums[1])
        assert padding_untouched(x)


@pytest.mark.parametrize("M,N", SIZES)
def test_gradient_that_overflows_over_x(M, N):
    """Infinities of dX in f16 stay there: dgamma and dbeta are of X and dY."""
    need_gpu()
    gen = torch.Generator().manual_seed(M)
    say(f"norm_grad over X {M}x{N}, dX past f16")
    x, dy = randn(gen, M, N, dtype="f16", scale=2.0 ** -9), randn(gen, M, N, dtype="f16", scale=2000.0)
    _, mean, rstd = norm(x, None, None, 0.0, "f16")
    dx, kept = out(M, N, dtype="f16"), x.clone()
    sums = grad(M, N, "f16", dy, x, None, mean, rstd, None, dx)
    check_grad(dy, kept, None, mean, rstd, None, "f16", None, *sums)
    assert torch.isinf(dx[M - 1]).any()
    over = grad(M, N, "f16", dy, x, None, mean, rstd, None, x)
    assert torch.equal(x, dx) and torch.equal(over[0], sums[0]) and torch.equal(over[1], sums[1])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("M,N", SIZES)
def test_norm_over_x(dtype, M, N):
    need_gpu()
    gen = torch.Generator().manual_seed(N)
    x, gamma, beta = randn(gen, M, N, dtype=dtype), randn(gen, 1, N, dtype=dtype)[0], randn(gen, 1, N, dtype=dtype)[0]
    want = norm(x.clone(), gamma, beta, 1e-5, dtype)
    got = norm(x, gamma, beta, 1e-5, dtype, inplace=True)
    assert got[0] is x and all(torch.equal(a, b) for a, b in zip(got, want))
