"""Output tiles of the products with 4-bit weights that one launch holds: 2^32 threads, by the tile that the call
takes. Pointers are fake addresses that the library only compares: a call of more is refused, and one of as many fails
at its launch where there is no GPU (and is left out where there is one)."""
import pytest
import torch

import dense_gemm_tile_amd as dgt

CALLS = [dgt._binding if hasattr(dgt, "_binding") else dgt._fast, dgt._CtypesCalls()]
A, B, S, Y, OFF = 1 << 50, 1 << 55, 1 << 56, 1 << 60, 1 << 57


def linear(M, N, K, group=128, ld=None):
    ld = ld or K
    return [c.gemm_linear_w4(M, N, K, "bf16", A, ld, B, 2 * ((ld + 1) // 2), S, None, (K + 127) // 128, group, None, "none", None, 0,
                             Y, N, "bf16", None) for c in CALLS]


def grouped(G, M, N, K):
    return [c.gemm_grouped_w4(G, M, N, K, "bf16", OFF, A, K, B, K, 0, S, None, (K + 127) // 128, 0, 128, None, "none", None, 0, Y, N,
                              "bf16", None) for c in CALLS]


# The most tiles of each: 384 threads and 64 x 64 (rows x columns), 448 and 64 x 32, 256 and 32 x 32 (through
# registers), 512 and 8 x 32 (one row of tiles); by rows 256 and 32 x 64, a tile more for each of 64 groups but
# for a row.
CASES = {
    "64x64": (lambda n: linear(64 * n, 64, 128), (2 ** 32 - 1) // 384),
    "64x64 wide": (lambda n: linear(128, 32 * n, 128), (2 ** 32 - 1) // 384),
    "64x32, groups of 32": (lambda n: linear(64 * n, 32, 32, group=32), (2 ** 32 - 1) // 448),
    "32x32": (lambda n: linear(32 * n, 32, 40, ld=41), (2 ** 32 - 1) // 256),
    "8x32": (lambda n: linear(8, 32 * n, 128), (2 ** 32 - 1) // 512),
    "32x64 by rows": (lambda n: grouped(64, 32 * (n - 62), 64, 128), (2 ** 32 - 1) // 256),
}


@pytest.mark.parametrize("name", list(CASES))
def test_more_tiles_than_a_launch_holds(name):
    call, most = CASES[name]
    if name == "64x64 wide":  # (two rows of tiles: an even number of them)
        most -= most % 2
    assert call(most + (2 if name == "64x64 wide" else 1)) == [dgt.GEMM_ERR_UNSUPPORTED] * 2
    assert "too many output tiles" in dgt.gemm_last_error()


@pytest.mark.parametrize("name", list(CASES))
def test_as_many_tiles_as_a_launch_holds(name):
    if torch.cuda.device_count():
        pytest.skip("would launch on addresses that are none")
    call, most = CASES[name]
    if name == "64x64 wide":
        most -= most % 2
    assert call(most) == [dgt.GEMM_ERR_HIP] * 2
    assert "launch failed" in dgt.gemm_last_error()


@pytest.mark.parametrize("M,N,K", [(8192, 151936, 4096), (65536, 16384, 4096)])
def test_large_ordinary_calls_are_not_refused(M, N, K):
    if torch.cuda.device_count():
        pytest.skip("would launch on addresses that are none")
    assert linear(M, N, K) == [dgt.GEMM_ERR_HIP] * 2
    assert grouped(64, 131072, 8192, 2048) == [dgt.GEMM_ERR_HIP] * 2
