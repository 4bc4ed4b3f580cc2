"""Products with 4-bit weights of many output tiles: calls as large as their own tiles let a launch be."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, U32, close, half_step, out, randn
from test_layer_w4_gpu import weights

pytestmark = pytest.mark.gpu


def rows_of(y, x, at, value, size, what):
    """Rows `at` of y against 64 bits: sums of K products, at most 31 + 16 times as large as the result's own."""
    want = x[at].double() @ value.T
    tol = (x.shape[1] + 16) * U32 * (x[at].double().abs() @ size.T)
    close(y[at], want, tol + half_step("bf16") * want.abs() + 1e-30, what)


@pytest.mark.parametrize("M,N,K", [(65536, 16384, 64), (8192, 151936, 32), (1200000, 1000, 40)])
def test_linear_of_many_tiles(M, N, K):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    say(f"linear_w4 {M}x{N}x{K}")
    gen = torch.Generator().manual_seed(1)
    c, s, z, value, size = weights(gen, (N,), K, 32, True, "bf16")
    x = torch.randn(M, K, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(torch.bfloat16)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    dgt.gemm_linear_w4(M, N, K, "bf16", x, K, c, 2 * c.stride(0), s, z, s.stride(0), 32, None, "none", None, 0, y, N, "bf16",
                       stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for lo in (0, M // 3, M - 70):
        rows_of(y, x, torch.arange(lo, lo + 70, device=DEV), value, size, dgt.gemm_last_path())


def test_experts_of_many_tiles():
    """A prompt's choices: 131072 rows for 64 experts, some without rows."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    G, M, N, K = 64, 131072, 8192, 32
    say(f"grouped_w4 {G} {M}x{N}x{K}")
    gen = torch.Generator().manual_seed(3)
    c, s, z, value, size = weights(gen, (G, N), K, 32, False, "bf16")
    x = torch.randn(M, K, device=DEV, generator=torch.Generator(DEV).manual_seed(4)).to(torch.bfloat16)
    counts = torch.rand(G, generator=gen) * (torch.rand(G, generator=gen) < 0.9)
    off = torch.nn.functional.pad((counts.cumsum(0) / counts.sum() * M).round().to(torch.int32), (1, 0)).to(DEV)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    dgt.gemm_grouped_w4(G, M, N, K, "bf16", off, x, K, c, 2 * c.stride(1), 2 * c.stride(0), s, z, s.stride(1), s.stride(0), 32,
                        None, "none", None, 0, y, N, "bf16", stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    ends = off.tolist()
    assert ends[-1] == M
    for g in range(G):
        if ends[g + 1] > ends[g]:
            at = torch.unique(torch.linspace(ends[g], ends[g + 1] - 1, 33).long()).to(DEV)
            rows_of(y, x, at, value[g], size[g], f"group {g}")
