"""Calls of more than 256 tiles on the 256x256 kernel, whose workgroups then walk several tiles each:
accumulators cleared between them, every tile found, and the LDS of one tile's epilogue filled again
by the next tile's operands."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import ACTS, close, half_step, ld, offsets_of, out, padding_untouched, randn, sum_tol, tiny
from test_layer_product_gpu import linear
from test_layer_tiles_gpu import tile

pytestmark = pytest.mark.gpu

# The contiguous dimensions fill whole tiles (the record count is the only mask); the others end
# inside one: 8 and 3 columns of the last column tile, so that most of its waves have none.
DENSE = [(0, 1, 4097, 4616, 64), (0, 1, 4097, 4616, 320), (0, 1, 4400, 4611, 192), (0, 0, 4097, 4864, 64),
         (0, 0, 4100, 4352, 192), (1, 0, 4352, 4352, 72), (1, 0, 4096, 4608, 200), (1, 1, 4352, 4616, 128)]


@pytest.mark.parametrize("tA,tB,M,N,K", DENSE)
def test_dense(tA, tB, M, N, K):
    need_gpu()
    assert -(-M // 256) * -(-N // 256) > 256
    gen = torch.Generator().manual_seed(M + N + K)
    with tile("pp256x256"):
        for i, kw in enumerate((dict(bias=True, residual=True, keep_z=True), dict(), dict(residual=True, r_is_y=True),
                                dict(bias=True, out_dtype="f32"))):
            path = linear(gen, M, N, K, ("bf16", "f16")[i % 2], tA, tB, act=ACTS[(i + K // 64) % 5], **kw)
            assert " pp256x256 " in path, path


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("f16", "f32")])
def test_grad_weight(dtype, out_dtype, accumulate):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(41 + accumulate)
    N, K, sizes = 1024, 2048, [64, 0, 1, 200, 65, 0, 130, 7, 63, 128, 0, 333]
    G, used = len(sizes), sum(sizes)
    assert G * (N // 256) * (K // 256) > 256
    say(f"grad_weight {sizes} N={N} K={K} {dtype}->{out_dtype} accumulate={accumulate}")
    M = used + 9
    a, b = randn(gen, M, N, dtype=dtype), randn(gen, M, K, dtype=dtype)
    a[used:], b[used:] = float("nan"), float("nan")
    d = out(G, N, K, dtype=out_dtype, pad=8)
    if accumulate:
        d.copy_(randn(gen, G, N, K, dtype=out_dtype))
    old = d.double().clone()
    with tile("pp256x256"):
        dgt.gemm_grouped_grad_weight(G, M, N, K, dtype, offsets_of(sizes), a, ld(a), b, ld(b), d, ld(d), d.stride(0),
                                     out_dtype, accumulate, stream=torch.cuda.current_stream())
    path = dgt.gemm_last_path()
    assert " pp256x256 " in path, path
    lo = 0
    for g, n in enumerate(sizes):
        s = slice(lo, lo + n)
        lo += n
        want = a[s].double().T @ b[s].double()
        tol = sum_tol(n, a[s].double().abs().T @ b[s].double().abs())
        if accumulate:
            want = want + old[g]
            tol = tol + 2.0 ** -24 * want.abs()
        close(d[g], want, tol * 1.01 + half_step(out_dtype) * want.abs() + tiny(out_dtype), f"group {g} {path}")
    assert padding_untouched(d)
