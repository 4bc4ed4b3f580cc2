"""Products with 4-bit weights against the values the codes stand for, in 64 bits."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import (ACTS, ACT_STEPS, DEV, DT, U32, act64, close, half_step, ld, offsets_of, out, padding_untouched,
                           randn, tiny)

pytestmark = pytest.mark.gpu


def weights(gen, shape, K, group, zeros, dtype, pad=0, fill=0xA7):
    """Codes [..., ldb / 2] bytes, scales and zero points [..., runs (+ pad)] and the values in 64 bits."""
    runs, width = -(-K // group), (K + 1) // 2
    q = torch.randint(0, 16, (*shape, 2 * width), generator=gen)
    codes = torch.full((*shape, width + pad), fill, dtype=torch.uint8)
    codes[..., :width] = (q[..., 0::2] | q[..., 1::2] << 4).to(torch.uint8)
    s = torch.full((*shape, runs + pad), float("nan"), dtype=DT[dtype])
    s[..., :runs] = ((0.5 + torch.rand(*shape, runs, generator=gen)) * 0.1).to(DT[dtype])
    z = None
    if zeros:
        z = torch.full_like(s, float("nan"))
        z[..., :runs] = (4 + 8 * torch.rand(*shape, runs, generator=gen)).to(DT[dtype])
    run = torch.arange(K) // group
    z64 = 8.0 if z is None else z.double()[..., run]
    w = s.double()[..., run] * (q[..., :K].double() - z64)
    mag = s.double()[..., run].abs() * (32 + q[..., :K].double() + z64)
    dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    return dev(codes), dev(s), dev(z), dev(w), dev(mag)


def want(x, w, mag, K, group, b, r, act, out_dtype):
    """Y and its tolerance. Each run's products of 16 + code, and its sum of values, are summed in
    float32 and scaled, and the runs are added: every rounding is at most half a step of the sum of
    absolute values |x| s (16 + code + 16 + zero)."""
    steps = min(group, K) + -(-K // group) + 16
    z, off = x @ w.T, steps * U32 * (x.abs() @ mag.T)
    if b is not None:
        z = z + b.double()
        off = off + 2 * U32 * z.abs()
    y = act64(z, act)
    tol = 1.2 * off + ACT_STEPS * U32 * y.abs()
    if r is not None:
        y = y + r.double()
        tol = tol + U32 * y.abs()
    return y, tol * (1 + half_step(out_dtype)) + half_step(out_dtype) * y.abs() + tiny(out_dtype)


def linear(gen, M, N, K, group, dtype, zeros=False, act="none", bias=False, residual=False, out_dtype=None, pad=0, wpad=0,
           inplace=False):
    import dense_gemm_tile_amd as dgt
    o = out_dtype or dtype
    say(f"w4 {M}x{N}x{K} group={group} {dtype}->{o} {zeros} {act} {bias} {residual} pad={pad},{wpad}")
    x = randn(gen, M, K, dtype=dtype, pad=pad)
    codes, s, z, w, mag = weights(gen, (N,), K, group, zeros, dtype, wpad)
    b = randn(gen, 1, N, dtype=dtype)[0] if bias else None
    r = randn(gen, M, N, dtype=o, pad=pad) if residual else None
    y64, tol = want(x.double(), w, mag, K, group, b, r, act, o)
    y = r if inplace else out(M, N, dtype=o, pad=pad)
    dgt.gemm_linear_w4(M, N, K, dtype, x, ld(x), codes, 2 * codes.stride(0), s, z, s.stride(0), group, b, act, r, ld(r), y,
                       ld(y), o, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    close(y, y64, tol, "Y")
    assert padding_untouched(y)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 256])
def test_linear_w4(dtype, group):
    need_gpu()
    gen = torch.Generator().manual_seed(group)
    for i, (M, N, K) in enumerate(((1, 1, 1), (1, 16, 32), (1, 40, 128), (2, 33, 260), (5, 64, 512), (16, 128, 1024),
                                   (17, 100, 384), (33, 72, 200), (48, 256, 640), (64, 130, 1000), (65, 48, 2048),
                                   (130, 96, 320), (1, 512, 4096), (300, 31, 77))):
        linear(gen, M, N, K, group, dtype, zeros=i % 2 == 0)
        linear(gen, M, N, K, group, dtype, zeros=i % 2 == 1, act=ACTS[i % 5], bias=True, residual=i % 3 == 0,
               out_dtype="f32" if i % 2 else None)


def test_linear_w4_row_ends_starts_and_pitches():
    """Every number of values past the last whole word, and rows of codes and values at any address."""
    need_gpu()
    gen = torch.Generator().manual_seed(3)
    for i in range(34):
        linear(gen, 1 + i, 20 + i, 1 + i, 32, "bf16", zeros=i % 2 == 0, pad=i % 4, wpad=i % 5)
        linear(gen, 3, 20 + i, 256 + 1 + i, 64, "f16", zeros=i % 2 == 1, pad=i % 3, wpad=(i + 1) % 7, out_dtype="f32")
        linear(gen, 70, 20, 127 + i, 128, "bf16", pad=1, wpad=i % 3, residual=True, inplace=i % 2 == 0)


@pytest.mark.parametrize("M,N,K,group,zeros,pad,path", [
    (1, 4096, 512, 128, True, 0, "w8 t8x16"), (8, 4112, 384, 64, False, 0, "w8 t8x32"), (9, 4112, 160, 32, True, 0, "w8 t16x32"),
    (31, 500, 2048, 32, True, 0, "w8 t32x32"), (47, 260, 1184, 64, True, 0, "w8 t48x32"), (64, 72, 1024, 96, True, 0, "w7 t64x32"),
    (130, 200, 640, 32, False, 0, "w7 t64x32"), (520, 1900, 384, 128, True, 0, "w6 t64x64"), (520, 1900, 256, 64, True, 0, "w7 t64x32"),
    (40, 64, 45056, 32, True, 0, "w8 t16x16"), (13, 300, 1000, 64, True, 1, "w8 t16x16 through registers"),
    (60, 200, 2100, 128, True, 1, "w8 t32x32 through registers"), (50, 130, 333, 96, False, 3, "w4 t16x32 through registers"),
    (1060, 1000, 200, 32, True, 1, "w4 t32x32 through registers"), (30, 50, 45057, 32, True, 0, "w8 t16x16 through registers")])
def test_every_tile(M, N, K, group, zeros, pad, path):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(M + N)
    for dtype in ("bf16", "f16"):
        linear(gen, M, N, K, group, dtype, zeros=zeros, act="silu", bias=True, residual=True, out_dtype="f32", pad=pad)
        assert dgt.gemm_last_path().endswith(path), dgt.gemm_last_path()


@pytest.mark.parametrize("sizes,N,K,group,zeros,path", [
    ([2, 0, 8, 5], 130, 1024, 128, False, "w4 t8x64"), ([2, 0, 8, 5], 130, 4096, 32, True, "w4 t8x32"),
    ([20, 0, 13], 130, 640, 64, True, "w4 t16x32"), ([50, 1, 70], 130, 640, 96, True, "w4 t32x64"),
    ([5, 0, 3], 40, 45056, 32, True, "w8 t16x16"), ([5, 0, 19], 40, 77, 32, True, "w8 t16x16 through registers"),
    ([60, 0, 30], 40, 2100, 128, False, "w8 t32x32 through registers"), ([60, 0, 30], 40, 90, 32, True, "w4 t16x32 through registers")])
def test_every_grouped_tile(sizes, N, K, group, zeros, path):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(N + K)
    for dtype in ("bf16", "f16"):
        grouped(gen, sizes, N, K, group, dtype, zeros=zeros, act="gelu", bias=True, residual=True, spare=2)
        assert dgt.gemm_last_path().endswith(path), dgt.gemm_last_path()


def test_linear_w4_without_a_sum_and_every_code():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    b = torch.arange(20, device=DEV).to(torch.bfloat16)
    y = out(3, 20, dtype="bf16")
    dgt.gemm_linear_w4(3, 20, 0, "bf16", None, 1, None, 2, None, None, 1, 32, b, "none", None, 0, y, 20, "bf16",
                       stream=torch.cuda.current_stream())
    assert torch.equal(y, b.expand(3, 20))
    for dtype in ("f16", "bf16"):
        # One weight at a time: the identity reads the whole matrix back, exactly.
        K = 96
        x = torch.eye(K, dtype=DT[dtype], device=DEV)
        codes = torch.arange(256, dtype=torch.uint8).repeat(3)[: 16 * K // 2].reshape(16, K // 2).to(DEV)
        s = torch.full((16, 3), 0.5, dtype=DT[dtype], device=DEV)
        s[:, 1], s[:, 2] = 2.0, -1.0
        y = out(K, 16)
        dgt.gemm_linear_w4(K, 16, K, dtype, x, K, codes, K, s, None, 3, 32, None, "none", None, 0, y, 16, "f32",
                           stream=torch.cuda.current_stream())
        q = torch.stack([codes & 15, codes >> 4], -1).reshape(16, K).double() - 8
        assert torch.equal(y.double(), (q * s.double().repeat_interleave(32, 1)).T)


def grouped(gen, sizes, N, K, group, dtype, zeros=False, act="none", bias=False, residual=False, out_dtype=None, spare=0,
            shared=False):
    import dense_gemm_tile_amd as dgt
    o, G, used = out_dtype or dtype, len(sizes), sum(sizes)
    M = used + spare
    say(f"grouped_w4 {sizes[:8]} {N}x{K} group={group} {dtype}->{o} {zeros} {act} {bias} spare={spare}")
    x = randn(gen, max(M, 1), K, dtype=dtype)[:M]
    codes, s, z, w, mag = weights(gen, (1 if shared else G, N), K, group, zeros, dtype)
    b = randn(gen, G, N, dtype=dtype) if bias else None
    r = randn(gen, M, N, dtype=o) if residual else None
    y = out(M, N, dtype=o)
    dgt.gemm_grouped_w4(G, M, N, K, dtype, offsets_of(sizes), x, K, codes, 2 * codes.stride(1),
                        0 if shared else 2 * codes.stride(0), s, z, s.stride(1), 0 if shared else s.stride(0), group, b, act,
                        r, ld(r), y, N, o, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    lo = 0
    for g, n in enumerate(sizes):
        part = slice(lo, lo + n)
        lo += n
        at = 0 if shared else g
        y64, tol = want(x[part].double(), w[at], mag[at], K, group, None if b is None else b[g],
                        None if r is None else r[part], act, o)
        close(y[part], y64, tol, f"group {g}")
    assert torch.isnan(y[used:]).all()


@pytest.mark.parametrize("sizes", [[0], [1], [3, 0, 5], [0, 0, 16, 0], [17, 1, 2, 64, 33], [2] * 20, [1, 0] * 40,
                                   [130, 0, 1], [0] * 5])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_grouped_w4(sizes, dtype):
    need_gpu()
    gen = torch.Generator().manual_seed(len(sizes))
    grouped(gen, sizes, 48, 256, 32, dtype, spare=3)
    grouped(gen, sizes, 33, 130, 64, dtype, zeros=True, act="silu", bias=True, residual=True)
    grouped(gen, sizes, 16, 512, 128, dtype, zeros=True, out_dtype="f32", spare=1, shared=True)


@pytest.mark.parametrize("K", [64, 40, 2100])
def test_offsets_of_another_program(K):
    """Offsets that decrease or pass the rows stay inside the buffers: rows past M are not there, and
    what lies around Y keeps its values."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(9)
    M, N, runs = 20, 40, -(-K // 32)
    x = randn(gen, M, K, dtype="bf16")
    codes, s, _, _, _ = weights(gen, (4, N), K, 32, False, "bf16")
    for off in ([0, 30, 10, 50, 20], [5, -7, 100, 3, 2 ** 31 - 1], [0, 0, 0, 0, 10 ** 6]):
        wide = out(M + 8, N, dtype="bf16")
        dgt.gemm_grouped_w4(4, M, N, K, "bf16", torch.tensor(off, dtype=torch.int32, device=DEV), x, K, codes, K, N * K, s,
                            None, runs, N * runs, 32, None, "none", None, 0, wide[4:], N, "bf16",
                            stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.isnan(wide[:4]).all() and torch.isnan(wide[-4:]).all()
