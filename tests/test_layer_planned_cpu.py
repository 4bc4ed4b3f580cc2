"""The kernel that grouped calls of few rows a group take when a row is not in whole 16-byte pieces, by
the expected number of 64 x 64 tiles rather than by the most that the groups' sizes could make. No GPU."""
import pytest

from test_layer_cpu import grouped, lib  # noqa: F401


def planned(lib, G, rows, N, K, tB, **kw):  # noqa: F811
    assert grouped(lib, G=G, M=G * rows, N=N, K=K, tB=tB, A=1 << 40, Y=1 << 50, **kw) == 0, lib.gemm_last_error()
    return lib.gemm_last_path().split()[2]


@pytest.mark.parametrize("tB", [1, 0])
@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 16, 32])
def test_many_tiles(lib, rows, tB):  # noqa: F811
    for G, N, K in ((64, 2048, 2048), (256, 1024, 512), (16, 4096, 1024), (128, 768, 768)):
        odd_a, odd_b = dict(lda=K + 1), dict(ldb=(K if tB else N) + 1, stride=2 * N * K)
        for kw in (odd_a, odd_b, odd_a | odd_b):
            assert planned(lib, G, rows, N, K, tB, **kw) == "g64x64", (G, N, K, kw)


@pytest.mark.parametrize("rows", [1, 2, 8, 16])
def test_few_tiles(lib, rows):  # noqa: F811
    for G, N, K in ((4, 1024, 1024), (8, 1024, 1024), (2, 4096, 4096)):
        assert planned(lib, G, rows, N, K, 1, lda=K + 1) == "u16x32"
        assert planned(lib, G, rows, N, K, 0, lda=K + 1) == "g64x64k4"
    for G, N, K in ((8, 2048, 2048), (64, 256, 4096), (12, 1024, 2048)):
        for tB in (0, 1):
            assert planned(lib, G, rows, N, K, tB, lda=K + 1) == "g64x64k4"


def test_more_rows_take_larger_tiles(lib):  # noqa: F811
    assert planned(lib, 64, 100, 2048, 2048, 1, lda=2049) == "g128x128"
    assert planned(lib, 64, 100, 2048, 2048, 0, ldb=2049, stride=2049 * 2048) == "r128x128"


def test_odd_weights_of_few_rows(lib):  # noqa: F811
    for G, N, K in ((24, 1024, 1024), (8, 4096, 2048), (8, 2048, 2048)):
        for rows, name in ((1, "u16x32"), (4, "u16x32"), (5, None)):
            got = planned(lib, G, rows, N, K, 1, ldb=K + 1, stride=2 * N * K)
            assert got == name or name is None and got != "u16x32"
