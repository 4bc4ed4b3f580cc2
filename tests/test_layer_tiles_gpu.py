"""Every product kernel of the layer operators, forced by name, at the edges of its tile: rows,
columns and sums that end inside it, groups smaller and larger than it, empty ones."""
import ctypes
from contextlib import contextmanager

import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import ACTS, close, half_step, ld, offsets_of, out, randn, sum_tol, tiny
from test_layer_product_gpu import grouped, linear

pytestmark = pytest.mark.gpu

LAYOUTS = [(0, 1), (0, 0), (1, 0), (1, 1)]
TILES = {"g128x128": (128, 128), "g64x64": (64, 64), "g64x64k4": (64, 64), "pp256x256": (256, 256), "pp128x128": (128, 128),
         "pp128x128deep": (128, 128)}
# A stored [M][K], those of ALL in any layout; s16x16 with B stored [N][K] only.
SKINNY = {"s16x32": (16, 32), "s32x32": (32, 32), "s64x32": (64, 32), "s64x64": (64, 64),
          "s16x16": (16, 16), "s48x32": (48, 32)}
ALL = ("s32x32", "s64x32", "s64x64")
NT_ONLY = ("s16x16", "r16x32")
# Any alignment and K, A stored [M][K], B stored [N][K].
ANY = {"u16x32": (16, 32), "u32x32": (32, 32), "u64x32": (64, 32)}


@contextmanager
def tile(name):
    env = ctypes.CDLL(None)
    env.setenv(b"GEMM_LAYER_TILE", name.encode(), 1)
    try:
        yield
    finally:
        env.unsetenv(b"GEMM_LAYER_TILE")


def layouts(name):
    return [la for la in LAYOUTS if name in TILES or name in ALL or (not la[0] and (la[1] or name not in NT_ONLY))]


@pytest.mark.parametrize("name", [*TILES, *SKINNY])
def test_dense_forced(name):
    need_gpu()
    bm, bn = {**TILES, **SKINNY}[name]
    gen = torch.Generator().manual_seed(bm * 5 + bn)
    i = 0
    with tile(name):
        for tA, tB in layouts(name):
            m_step = 8 if tA else 1  # A stored [K][M] has to hold whole 16-byte pieces
            for M, N in ((m_step, 8), (bm, bn), (bm - 3 * m_step, bn + 8), (2 * bm + m_step, 3 * bn - 8)):
                if M < 1:
                    continue
                for K in (8, 56, 64, 72, 128, 200, 328, 584, 1096, 2056):
                    dtype = ("f16", "bf16")[i % 2]
                    path = linear(gen, M, N, K, dtype, tA, tB, act=ACTS[i % 5], bias=i % 2 == 0,
                                  residual=i % 3 == 0, keep_z=i % 4 == 1, out_dtype="f32" if i % 3 == 1 else dtype,
                                  pads=(0, 0, 0) if i % 3 else (8, 16, 8))
                    assert f" {name} " in path, path
                    i += 1


@pytest.mark.parametrize("name", [*TILES, *SKINNY, "r16x32"])
def test_grouped_forced(name):
    need_gpu()
    bm, bn = {**TILES, **SKINNY, "r16x32": (16, 32)}[name]
    gen = torch.Generator().manual_seed(bm * 3 + bn)
    sizes = [[1], [0, 0, bm, 0], [bm - 1, 1, bm + 1, 0, 3 * bm + 5], [1, 0, 2] * 30, [0], [7] * 67, [bm] * 3]
    with tile(name):
        for tA, tB in layouts(name):
            if tA:
                continue
            for i, s in enumerate(sizes):
                for N, K in ((bn, 64), (bn + 8, 136), (8, 648)):
                    path = grouped(gen, s, N, K, ("f16", "bf16")[i % 2], tB, act=ACTS[i % 5], bias=i % 2 == 0,
                                   residual=i % 3 == 0, keep_z=i % 4 == 1, spare=(i * 7) % 20,
                                   out_dtype="f32" if i % 3 == 1 else None, shared=i == 3)
                    assert f" {name} " in path, path


@pytest.mark.parametrize("name", list(ANY))
def test_any_alignment_forced(name):
    need_gpu()
    bm, bn = ANY[name]
    gen = torch.Generator().manual_seed(bm * 11 + bn)
    i = 0
    with tile(name):
        for pads in ((0, 0, 0), (1, 0, 3), (0, 1, 0), (3, 5, 1), (2, 4, 6)):
            for M, N in ((1, 1), (bm, bn), (bm - 3, bn + 3), (2 * bm + 1, 3 * bn - 5)):
                for K in (1, 2, 7, 8, 9, 63, 64, 65, 129, 520, 701, 1033, 2055):
                    dtype = ("f16", "bf16")[i % 2]
                    path = linear(gen, M, N, K, dtype, 0, 1, act=ACTS[i % 5], bias=i % 2 == 0, residual=i % 3 == 0,
                                  keep_z=i % 4 == 1, out_dtype="f32" if i % 3 == 1 else dtype, pads=pads)
                    assert f" {name} " in path, path
                    i += 1
        for i, s in enumerate([[1], [0, 0, bm, 0], [bm - 1, 1, bm + 1, 0, 3 * bm + 5], [1, 0, 2] * 30]):
            for N, K in ((bn + 1, 65), (7, 701), (bn, 128)):
                path = grouped(gen, s, N, K, ("f16", "bf16")[i % 2], 1, act=ACTS[i % 5], bias=i % 2 == 0,
                               keep_z=i % 4 == 1, spare=(i * 7) % 20, pads=(i % 3, i % 2, 0))
                assert f" {name} " in path, path


@pytest.mark.parametrize("tA,tB", [(0, 0), (1, 0), (1, 1)])
def test_staged_ring_forced(tA, tB):
    """Operands not stored along K with odd widths, pitches and starts; the others aligned."""
    need_gpu()
    gen = torch.Generator().manual_seed(21 + 2 * tA + tB)
    along_k = not tA or tB  # some operand is stored along K: whole pieces of it
    i = 0
    with tile("r128x128"):
        for pad in (0, 1, 2, 5, 8):
            pads = (pad if tA else 8 * (pad % 2), 8 * (pad % 2) if tB else pad, (0, 3, 8)[i % 3])
            for M, N in ((1, 1), (128, 128), (125, 131), (259, 391), (7, 300)):
                for K in (1, 8, 63, 64, 65, 72, 200, 333, 1096):
                    if along_k and K % 8:
                        continue
                    dtype = ("f16", "bf16")[i % 2]
                    path = linear(gen, M, N, K, dtype, tA, tB, act=ACTS[i % 5], bias=i % 2 == 0, residual=i % 3 == 0,
                                  keep_z=i % 4 == 1, out_dtype="f32" if i % 3 == 1 else dtype, pads=pads)
                    assert " r128x128 " in path, path
                    i += 1
        if not tA:
            for i, s in enumerate([[1], [0, 0, 128, 0], [127, 1, 129, 0, 389], [1, 0, 2] * 30]):
                for N, K in ((129, 72), (7, 704), (128, 128)):
                    path = grouped(gen, s, N, K, ("f16", "bf16")[i % 2], 0, act=ACTS[i % 5], bias=i % 2 == 0,
                                   keep_z=i % 4 == 1, spare=(i * 7) % 20, pads=(0, i % 4, i % 3))
                    assert " r128x128 " in path, path


def test_any_alignment_of_the_first_element():
    """Operands that start 2, 4, 6 ... bytes into an allocation, odd pitches."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    from layer_helpers import linear_want
    gen = torch.Generator().manual_seed(12)
    for name, (bm, _) in ANY.items():
        with tile(name):
            for ao in range(4):
                for bo in range(4):
                    M, N, K, lda, ldb = bm + 1, 37, 203, 203 + ao, 203 + bo
                    x = randn(gen, (M + 1) * lda, dtype="bf16")[ao:]
                    w = randn(gen, (N + 1) * ldb, dtype="bf16")[bo:]
                    xs = torch.as_strided(x, (M, K), (lda, 1), x.storage_offset())
                    ws = torch.as_strided(w, (N, K), (ldb, 1), w.storage_offset())
                    y = out(M, N, dtype="f32")
                    say(f"{name} starts {2 * ao} and {2 * bo} bytes in")
                    dgt.gemm_linear(M, N, K, "bf16", 0, 1, xs, lda, ws, ldb, None, "none", None, 0, y, N, "f32",
                                    stream=torch.cuda.current_stream())
                    wy, _, ty, _ = linear_want(xs, ws.T, None, None, "none", "bf16", "f32")
                    close(y, wy, ty, dgt.gemm_last_path())


@pytest.mark.parametrize("name", [*TILES, *ALL, "r128x128"])
def test_grad_weight_forced(name):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    bm, bn = {**TILES, **SKINNY, "r128x128": (125, 131)}[name]
    gen = torch.Generator().manual_seed(bm + bn)
    with tile(name):
        for i, sizes in enumerate([[1], [0], [64, 0, 65], [200, 1, 0, 63, 330], [3, 0] * 20]):
            for N, K in ((bm, bn), (bm + 8, bn - 8), (8, 2 * bn + 8)):
                dtype, out_dtype = ("f16", "bf16")[i % 2], ("f32", None)[i % 2]
                out_dtype = out_dtype or dtype
                say(f"grad_weight {sizes[:8]} N={N} K={K} {dtype}->{out_dtype}")
                G, used = len(sizes), sum(sizes)
                M = used + 5
                a, b = randn(gen, M, N, dtype=dtype), randn(gen, M, K, dtype=dtype)
                a[used:], b[used:] = float("nan"), float("nan")
                d = randn(gen, G, N, K, dtype=out_dtype)
                old = d.double().clone()
                dgt.gemm_grouped_grad_weight(G, M, N, K, dtype, offsets_of(sizes), a, ld(a), b, ld(b), d, ld(d),
                                             d.stride(0), out_dtype, i % 2, stream=torch.cuda.current_stream())
                path = dgt.gemm_last_path()
                assert f" {name} " in path, path
                lo = 0
                for g, n in enumerate(sizes):
                    s = slice(lo, lo + n)
                    lo += n
                    want = a[s].double().T @ b[s].double()
                    tol = sum_tol(n, a[s].double().abs().T @ b[s].double().abs())
                    if i % 2:
                        want = want + old[g]
                        tol = tol + 2.0 ** -24 * want.abs()
                    close(d[g], want, tol * 1.01 + half_step(out_dtype) * want.abs() + tiny(out_dtype),
                          f"group {g} {path}")


@pytest.mark.parametrize("name", ["pp256x256", "pp128x128", "s16x32"])
def test_refused_where_rows_are_not_16_byte_pieces(name):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(1)
    x, w, y = randn(gen, 8, 65, dtype="f16"), randn(gen, 8, 65, dtype="f16"), out(8, 8, dtype="f16")
    with tile(name), pytest.raises(dgt.GemmError):
        dgt.gemm_linear(8, 8, 65, "f16", 0, 1, x, 65, w, 65, None, "none", None, 0, y, 8, "f16",
                        stream=torch.cuda.current_stream())
