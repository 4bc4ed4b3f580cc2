"""Sizes at the edge of what a launch or 64-bit arithmetic holds: refused before anything is enqueued.
No GPU: every call here is refused or only checked."""
import ctypes

import pytest

from test_layer_cpu import A0, B0, P0, R0, W0, Y0, Z0, act_grad, call, grad_weight, grouped, lib, linear  # noqa: F401

MOST = 2 ** 31 - 1024


def test_tiles_of_a_launch(lib):  # noqa: F811
    # 512 threads a workgroup: 2^23 - 1 tiles of 16 rows and 32 columns, one row of tiles a group
    env = ctypes.CDLL(None)
    env.setenv(b"GEMM_LAYER_TILE", b"u16x32", 1)
    try:
        assert grouped(lib, G=32767, M=32767, N=256 * 32, K=65, lda=65, ldb=65, stride=0, Y=1 << 60) == 0
        assert " u16x32 " in lib.gemm_last_path()
        assert grouped(lib, G=32768, M=32768, N=256 * 32, K=65, lda=65, ldb=65, stride=0, Y=1 << 60) == 2
        assert "too many" in lib.gemm_last_error()
    finally:
        env.unsetenv(b"GEMM_LAYER_TILE")
    # the longest dense calls still fit
    assert linear(lib, M=MOST, N=1, K=1, A=A0, B=1 << 56, Y=1 << 60) == 0
    assert linear(lib, M=MOST, N=8, K=8, A=A0, B=1 << 56, Y=1 << 60) == 0


def test_pieces_of_rows(lib):  # noqa: F811
    assert call(lib, "gemm_combine", MOST, 1, 200, 1, A0, 201, 1 << 50, None, None, 0, 1 << 60, 201, None) == 2
    assert "too many" in lib.gemm_last_error()
    M, N = 1 << 24, 1 << 22  # 2^19 times 2^13 waves
    big = dict(M=M, N=N, lddy=N, ldz=N, lddz=N, Z=1 << 55, dZ=1 << 56, db=None)
    assert act_grad(lib, **big) == 2
    assert "too many" in lib.gemm_last_error()


@pytest.mark.parametrize("ldd,stride", [(1 << 33, 0), (1 << 33, 1 << 62), (1 << 40, 1 << 50), (1 << 62, (1 << 63) - 1)])
def test_overlapping_weight_gradients_of_far_rows(lib, ldd, stride):  # noqa: F811
    """One matrix is (N - 1) * ldd + K elements, which 64 bits need not hold."""
    assert grad_weight(lib, G=2, N=MOST, K=8, lda=MOST, M=0, A=None, B=None, D=1 << 40, ldd=ldd, stride=stride) == 1
    assert "stride_d" in lib.gemm_last_error()
