"""Joining rows in calls large enough for the kernels that take two pieces a lane, and, from 128 MiB of
rows on, for those that ask the caches to keep nothing: against the definition in 64 bits."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import U32, close, half_step, ld, out, padding_untouched, randn, tiny
from test_layer_rows_gpu import slots

pytestmark = pytest.mark.gpu

SIZE = {"f16": 2, "bf16": 2, "f32": 4}
# T, top, H, type, padding of rows. Two pieces a lane: T * H of at least 2^19 elements for each
# element of an access, which H and the padding make 8 (f32: 4), 4, 2 or 1.
TWO = [(4200, 2, 1032, "bf16", 0), (4200, 3, 1032, "f16", 8), (2200, 2, 1028, "bf16", 4), (1100, 2, 1030, "f16", 2),
       (600, 5, 1031, "bf16", 1), (520, 2, 1033, "f16", 0), (2200, 2, 1028, "f32", 0), (1100, 1, 1030, "f32", 2),
       (600, 2, 1031, "f32", 1), (270000, 2, 8, "f32", 0), (530000, 1, 8, "bf16", 0)]
ONCE = [(4100, 4, 4104, "bf16", 0), (4100, 4, 4103, "f16", 0), (4100, 4, 4100, "f16", 2), (4100, 5, 4102, "bf16", 1),
        (2100, 4, 4004, "f32", 0), (2100, 4, 4002, "f32", 1), (1100000, 8, 8, "bf16", 0), (70000, 8, 130, "f16", 6)]


def combine(gen, T, top, H, dtype, pad, drop, weights, residual):
    import dense_gemm_tile_amd as dgt
    say(f"combine {T}x{top}x{H} {dtype} pad={pad} drop={drop} weights={weights} residual={residual}")
    slot, n = slots(gen, T, top, drop), T * top
    kept = (slot >= 0) & (slot < n)
    ys = randn(gen, n, H, dtype=dtype, pad=pad)
    w = randn(gen, T, top) if weights else None
    r = randn(gen, T, H, dtype=dtype, pad=pad) if residual else None
    y = out(T, H, dtype=dtype, pad=pad)
    if residual == "in place":
        y.copy_(r)
    rin = y if residual == "in place" else r
    dgt.gemm_combine(T, top, H, dtype, ys, ld(ys), slot, w, rin, ld(rin), y, ld(y),
                     stream=torch.cuda.current_stream())
    assert padding_untouched(y)
    step = max(1, 2 ** 23 // (top * H))  # tokens at a time
    for lo in range(0, T, step):
        t = slice(lo, lo + step)
        share = (w[t].double() if weights else 1.0) * kept[t]
        rows = ys[slot[t].clamp(0, n - 1).long()].double() * share[:, :, None]
        want, mag = rows.sum(1), rows.abs().sum(1)
        if residual:
            want, mag = want + r[t].double(), mag + r[t].double().abs()
        close(y[t], want, (top + 2) * U32 * mag * 1.01 + half_step(dtype) * want.abs() + tiny(dtype), f"Y from {lo}")


@pytest.mark.parametrize("T,top,H,dtype,pad", TWO)
def test_two_pieces_a_lane(T, top, H, dtype, pad):
    need_gpu()
    piece = 16 // SIZE[dtype]
    while H % piece or (H + pad) % piece:
        piece //= 2
    assert T * H >= 2 ** 19 * piece and T * top * H * SIZE[dtype] < 2 ** 27
    gen = torch.Generator().manual_seed(81)
    combine(gen, T, top, H, dtype, pad, 0.2, True, "in place")
    combine(gen, T, top, H, dtype, pad, 0.0, False, None)


@pytest.mark.parametrize("T,top,H,dtype,pad", ONCE)
def test_rows_read_once(T, top, H, dtype, pad):
    need_gpu()
    assert T * top * H * SIZE[dtype] >= 2 ** 27
    gen = torch.Generator().manual_seed(82)
    combine(gen, T, top, H, dtype, pad, 0.2, True, "in place")
    combine(gen, T, top, H, dtype, pad, 0.05, False, "apart")
