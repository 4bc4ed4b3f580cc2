"""Offsets that break their contract: they decrease, are negative or lie past the rows. What the calls
compute is then not defined, but they end, write only inside their outputs, and the next call on
proper offsets is right."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, randn
from test_layer_product_gpu import grouped
from test_layer_tiles_gpu import ANY, SKINNY, TILES, tile

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
# G + 1 offsets each; rows: 300
BROKEN = [[300, 0], [0, 300, 0, 300, 0, 300], [-5, -1, 20, 19, 18, 300], [BIG, -BIG - 1, BIG, 7], [0, 400, 500, 600],
          [i * 7919 % 601 - 150 for i in range(200)], [-BIG - 1] * 70 + [BIG] * 70, [0, 300] * 100]
GUARD = 4096  # elements on both sides of an output


def guarded(*shape, dtype=torch.bfloat16):
    """A zeroed matrix and the words around it, which no call may change."""
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + 2 * GUARD,), 77.0, dtype=dtype, device=DEV)
    whole[GUARD:GUARD + n] = 0
    return whole[GUARD:GUARD + n].view(*shape), whole


def untouched(whole):
    return bool((whole[:GUARD] == 77).all() and (whole[-GUARD:] == 77).all())


def tensor(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("name", [*TILES, *SKINNY, "r16x32", *ANY, "r128x128"])
def test_grouped(name):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(61)
    M, N, K = 300, 136, 264
    tB = 0 if name == "r128x128" else 1
    with tile(name):
        for offsets in BROKEN:
            G = len(offsets) - 1
            say(f"{name} offsets {offsets[:8]} of {G} groups")
            x = randn(gen, M, K, dtype="bf16")
            w = randn(gen, G, *((N, K) if tB else (K, N)), dtype="bf16")
            y, ywhole = guarded(M, N)
            z, zwhole = guarded(M, N)
            dgt.gemm_grouped(G, M, N, K, "bf16", tB, tensor(offsets), x, K, w, w.stride(1), w.stride(0), None, "silu",
                             None, 0, y, N, "bf16", z, N, stream=torch.cuda.current_stream())
            torch.cuda.synchronize()
            assert f" {name} " in dgt.gemm_last_path()
            assert untouched(ywhole) and untouched(zwhole)
        grouped(gen, [5, 0, 130, 17], N, K, "bf16", tB, act="silu")


def test_act_grad_and_grad_weight():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(62)
    M, N, K = 300, 136, 72
    s = torch.cuda.current_stream()
    for offsets in BROKEN:
        G = len(offsets) - 1
        say(f"offsets {offsets[:8]} of {G} groups")
        dy, z, off = randn(gen, M, N, dtype="f16"), randn(gen, M, N, dtype="f16"), tensor(offsets)
        dz, dzw = guarded(M, N, dtype=torch.float16)
        db, dbw = guarded(G, N, dtype=torch.float32)
        size = dgt.gemm_act_grad_workspace(G, M, N)
        ws, wsw = guarded(size // 4, dtype=torch.float32)
        dgt.gemm_act_grad(G, M, N, "f16", "gelu", off, dy, N, z, N, dz, N, db, ws, size, stream=s)
        dw, dww = guarded(G, N, K, dtype=torch.float32)
        dgt.gemm_grouped_grad_weight(G, M, N, K, "f16", off, dy, N, randn(gen, M, K, dtype="f16"), K, dw, K, N * K,
                                     "f32", stream=s)
        torch.cuda.synchronize()
        for w in (dzw, dbw, wsw, dww):
            assert untouched(w)


@pytest.mark.parametrize("name", ["s16x32", "u16x32"])
def test_more_tiles_than_32_bits_count(name):
    """2047 groups, every other one of all rows: 1024 times 4100 row tiles of 1024 column tiles are
    2^32 and four million more."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(63)
    M, N, K, G = 65600, 32768, 64, 2047
    say(f"{name} {G} groups of {M} and 0 rows in turn")
    x, w = randn(gen, M, K, dtype="bf16"), randn(gen, N, K, dtype="bf16")
    y, whole = guarded(M, N)
    off = tensor([0, M]).repeat((G + 1) // 2)
    with tile(name):
        dgt.gemm_grouped(G, M, N, K, "bf16", 1, off, x, K, w, K, 0, None, "none", None, 0, y, N, "bf16",
                         stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert f" {name} " in dgt.gemm_last_path()
    assert untouched(whole)
    grouped(gen, [5, 0, 130, 17], 136, 264, "bf16", 1)
