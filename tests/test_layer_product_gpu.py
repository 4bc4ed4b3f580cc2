"""The layer operators' products against their definition in 64 bits: fused linear layers, one
weight matrix per group of rows, and the gradient of those weights."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import (ACTS, DEV, close, half_step, ld, linear_want, offsets_of, out,
                           padding_untouched, randn, sum_tol, tiny)

pytestmark = pytest.mark.gpu


def linear(gen, M, N, K, dtype, tA, tB, *, act="none", bias=False, residual=False, keep_z=False,
           out_dtype=None, pads=(0, 0, 0), r_is_y=False, stream=None):
    import dense_gemm_tile_amd as dgt
    out_dtype = out_dtype or dtype
    say(f"linear {M}x{N}x{K} {dtype}->{out_dtype} tA={tA} tB={tB} act={act} b={bias} r={residual} "
        f"z={keep_z} pads={pads}")
    x = randn(gen, *((K, M) if tA else (M, K)), dtype=dtype, pad=pads[0])
    w = randn(gen, *((N, K) if tB else (K, N)), dtype=dtype, pad=pads[1], scale=max(K, 1) ** -0.5)
    b = randn(gen, N, dtype=dtype) if bias else None
    r = randn(gen, M, N, dtype=out_dtype, pad=pads[2]) if residual else None
    y = out(M, N, dtype=out_dtype, pad=pads[2])
    if r_is_y:
        y.copy_(r)
    z = out(M, N, dtype=dtype, pad=pads[2]) if keep_z else None
    rin = y if r_is_y else r
    dgt.gemm_linear(M, N, K, dtype, tA, tB, x, ld(x), w, ld(w), b, act, rin, ld(rin), y, ld(y),
                    out_dtype, z, ld(z), stream=stream or torch.cuda.current_stream())
    path = dgt.gemm_last_path()
    torch.cuda.synchronize()
    wy, wz, ty, tz = linear_want(x.T if tA else x, w.T if tB else w, b, r, act, dtype, out_dtype)
    close(y, wy, ty, f"Y {path}")
    assert padding_untouched(y)
    if keep_z:
        close(z, wz, tz, f"Z {path}")
        assert padding_untouched(z)
    return path


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 256, 1024), (3, 5, 7), (2, 8, 4096), (16, 48, 136), (17, 33, 65),
          (33, 96, 264), (64, 64, 64), (65, 520, 128), (128, 128, 192), (130, 200, 72), (200, 1000, 520),
          (257, 129, 1032), (256, 512, 64), (300, 264, 200)]


@pytest.mark.parametrize("tA,tB", [(0, 1), (0, 0), (1, 0), (1, 1)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linear_shapes(dtype, tA, tB):
    need_gpu()
    gen = torch.Generator().manual_seed(100 + 2 * tA + tB)
    for i, (M, N, K) in enumerate(SHAPES):
        linear(gen, M, N, K, dtype, tA, tB, act=ACTS[i % 5], bias=i % 2 == 0, residual=i % 3 == 0,
               keep_z=i % 4 == 1, out_dtype="f32" if i % 3 == 1 else dtype)


@pytest.mark.parametrize("pads", [(8, 16, 8), (1, 0, 0), (0, 3, 1), (2, 4, 6), (0, 0, 5)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linear_pitches(dtype, pads):
    need_gpu()
    gen = torch.Generator().manual_seed(31)
    for tA, tB in ((0, 1), (0, 0), (1, 0), (1, 1)):
        linear(gen, 130, 72, 264, dtype, tA, tB, act="silu", bias=True, residual=True, keep_z=True,
               pads=pads)
        linear(gen, 7, 136, 520, dtype, tA, tB, act="gelu", bias=True, residual=True, pads=pads,
               out_dtype="f32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_linear_epilogue(act, out_dtype):
    need_gpu()
    gen = torch.Generator().manual_seed(5)
    for bias in (False, True):
        for residual in (False, True):
            linear(gen, 70, 136, 96, "bf16", 0, 1, act=act, bias=bias, residual=residual,
                   keep_z=residual, out_dtype=out_dtype)
    linear(gen, 70, 136, 96, "bf16", 0, 1, act=act, residual=True, r_is_y=True, out_dtype=out_dtype)


@pytest.mark.parametrize("M,N,K,tA,tB", [(1, 4096, 4096, 0, 1), (5, 1000, 2048, 0, 1), (31, 2048, 1032, 0, 1),
                                         (48, 4096, 2048, 0, 1), (96, 8192, 1024, 0, 1), (4, 2048, 4096, 0, 0),
                                         (512, 2048, 2048, 0, 1), (1024, 1024, 4096, 0, 0),
                                         (1024, 1000, 4097, 1, 0), (2048, 4096, 512, 0, 1), (2300, 2048, 1000, 0, 1),
                                         (4097, 1000, 1032, 0, 1), (4096, 4096, 1024, 0, 1), (4000, 4104, 520, 0, 0),
                                         (4096, 4096, 520, 1, 0), (4104, 4096, 333, 1, 0)])
def test_linear_large(M, N, K, tA, tB):
    need_gpu()
    gen = torch.Generator().manual_seed(M + K)
    linear(gen, M, N, K, "bf16", tA, tB, act="gelu", bias=True, residual=True, keep_z=True)
    linear(gen, M, N, K, "f16", tA, tB, act="none", out_dtype="f32")


def test_linear_without_a_sum_is_the_bias():
    need_gpu()
    gen = torch.Generator().manual_seed(8)
    linear(gen, 5, 24, 0, "bf16", 0, 1, act="silu", bias=True, residual=True, keep_z=True)
    linear(gen, 5, 24, 0, "f16", 0, 0, act="gelu")


def test_linear_specials():
    """Infinities and NaN in one row and one column reach exactly that row and column."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(9)
    M, N, K = 40, 72, 136
    x, w = randn(gen, M, K, dtype="bf16"), randn(gen, N, K, dtype="bf16")
    x[3, 5], x[7, 0], w[11, 9] = float("inf"), float("nan"), float("nan")
    for act in ("none", "relu"):
        y = out(M, N, dtype="f32")
        dgt.gemm_linear(M, N, K, "bf16", 0, 1, x, K, w, K, None, act, None, 0, y, N, "f32",
                        stream=torch.cuda.current_stream())
        wy, _, ty, _ = linear_want(x, w.T, None, None, act, "bf16", "f32")
        nan = torch.isnan(x.double() @ w.T.double())
        wy = torch.where(nan, torch.full_like(wy, float("nan")), wy)
        close(y, wy, torch.nan_to_num(ty), act)


def test_linear_activation_range():
    """Activations far from zero: one product each, so Y is act() of a known number."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    v = torch.cat([torch.linspace(-30, 30, 601), torch.tensor([-1e4, -300.0, -90.0, 90.0, 300.0, 3e4]),
                   torch.tensor([-3e38, 3e38, 1e20, -1e20])]).to(torch.bfloat16).to(DEV)
    x = v[:, None].contiguous()
    w = torch.ones(1, 1, dtype=torch.bfloat16, device=DEV)
    for act in ACTS:
        y = out(len(v), 1, dtype="f32")
        dgt.gemm_linear(len(v), 1, 1, "bf16", 0, 1, x, 1, w, 1, None, act, None, 0, y, 1, "f32",
                        stream=torch.cuda.current_stream())
        wy, _, ty, _ = linear_want(x, w.T, None, None, act, "bf16", "f32")
        wy = torch.nan_to_num(wy, nan=0.0)  # z^3 overflows nothing in 64 bits; 0 * inf does not arise
        # values below float32's normal range may come out as zero
        close(y, wy, ty + 2.0 ** -126 * v.double().abs().clamp(min=1)[:, None], act)


GROUPS = [[1], [0], [5, 0, 3], [0, 0, 64, 0], [64, 128, 1, 31, 200], [300], [17] * 9, [1, 0, 0, 2] * 20,
          [256, 255, 257, 0, 3], [2, 0] * 70]


def grouped(gen, sizes, N, K, dtype, tB, *, act="none", bias=False, residual=False, keep_z=False,
            out_dtype=None, spare=0, pads=(0, 0, 0), shared=False):
    import dense_gemm_tile_amd as dgt
    out_dtype = out_dtype or dtype
    G, used = len(sizes), sum(sizes)
    M = used + spare
    say(f"grouped {sizes[:8]} N={N} K={K} {dtype}->{out_dtype} tB={tB} act={act} spare={spare}")
    x = randn(gen, M, K, dtype=dtype, pad=pads[0])
    x[used:] = float("nan")
    w = randn(gen, 1 if shared else G, *((N, K) if tB else (K, N)), dtype=dtype, pad=pads[1],
              scale=K ** -0.5)
    b = randn(gen, G, N, dtype=dtype) if bias else None
    r = randn(gen, M, N, dtype=out_dtype, pad=pads[2]) if residual else None
    y, z = out(M, N, dtype=out_dtype, pad=pads[2]), out(M, N, dtype=dtype, pad=pads[2]) if keep_z else None
    dgt.gemm_grouped(G, M, N, K, dtype, tB, offsets_of(sizes), x, ld(x), w, ld(w),
                     0 if shared else w.stride(0), b, act, r, ld(r), y, ld(y), out_dtype, z, ld(z),
                     stream=torch.cuda.current_stream())
    path = dgt.gemm_last_path()
    torch.cuda.synchronize()
    lo = 0
    for g, n in enumerate(sizes):
        s = slice(lo, lo + n)
        lo += n
        wg = w[0 if shared else g]
        wy, wz, ty, tz = linear_want(x[s], wg.T if tB else wg, b[g] if bias else None,
                                     r[s] if residual else None, act, dtype, out_dtype)
        close(y[s], wy, ty, f"Y of group {g} {path}")
        if keep_z:
            close(z[s], wz, tz, f"Z of group {g} {path}")
    assert torch.isnan(y[used:]).all() and padding_untouched(y)
    assert z is None or torch.isnan(z[used:]).all()
    return path


@pytest.mark.parametrize("tB", [1, 0])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_grouped(dtype, tB):
    need_gpu()
    gen = torch.Generator().manual_seed(200 + tB)
    for i, sizes in enumerate(GROUPS):
        for N, K in ((64, 64), (136, 200), (33, 65)):
            grouped(gen, sizes, N, K, dtype, tB, act=ACTS[i % 5], bias=i % 2 == 0, residual=i % 3 == 0,
                    keep_z=i % 4 == 1, out_dtype="f32" if i % 3 == 1 else dtype, spare=(i * 7) % 20)


@pytest.mark.parametrize("tB", [1, 0])
def test_grouped_large(tB):
    need_gpu()
    gen = torch.Generator().manual_seed(77)
    grouped(gen, [700, 0, 1300, 20, 513, 1], 1024, 512, "bf16", tB, act="gelu", bias=True, keep_z=True, spare=9)
    grouped(gen, [2100, 1900, 3000, 1192], 2048, 1000, "f16", tB, act="silu", bias=True)
    grouped(gen, [3, 1, 0, 7, 2] * 13, 2048, 1024, "bf16", tB, act="silu")
    grouped(gen, [40, 10, 90, 60] * 8, 512, 2048, "bf16", tB, out_dtype="f32", residual=True)
    grouped(gen, [130, 7], 72, 264, "f16", tB, pads=(1, 3, 5), bias=True)
    grouped(gen, [13, 70, 0, 4], 136, 96, "bf16", tB, shared=True, bias=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_weight(dtype, accumulate):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(300)
    big = [([700, 0, 1300, 20, 513, 1], 1024, 512), ([2100, 900], 1000, 2056), ([600] * 8, 768, 1024)]
    for i, (sizes, N, K) in enumerate([(s, n, k) for s in GROUPS for n, k in ((64, 64), (136, 200), (33, 65))] + big):
        out_dtype = "f32" if i % 2 else dtype
        spare, pad = (i * 5) % 12, (0, 0, 8, 3)[i % 4]
        G, used = len(sizes), sum(sizes)
        M = used + spare
        say(f"grad_weight {sizes[:8]} N={N} K={K} {dtype}->{out_dtype} pad={pad}")
        a, b = randn(gen, M, N, dtype=dtype, pad=pad), randn(gen, M, K, dtype=dtype, pad=pad)
        a[used:], b[used:] = float("nan"), float("nan")
        d = out(G, N, K, dtype=out_dtype, pad=pad)
        if accumulate:
            d.copy_(randn(gen, G, N, K, dtype=out_dtype))
        old = d.double().clone()
        dgt.gemm_grouped_grad_weight(G, M, N, K, dtype, offsets_of(sizes), a, ld(a), b, ld(b), d, ld(d),
                                     d.stride(0), out_dtype, accumulate,
                                     stream=torch.cuda.current_stream())
        path = dgt.gemm_last_path()
        lo = 0
        for g, n in enumerate(sizes):
            s = slice(lo, lo + n)
            lo += n
            want = a[s].double().T @ b[s].double()
            tol = sum_tol(n, a[s].double().abs().T @ b[s].double().abs())
            if accumulate:
                want = want + old[g]
                tol = tol + 2.0 ** -24 * want.abs()
            close(d[g], want, tol * 1.01 + half_step(out_dtype) * want.abs() + tiny(out_dtype),
                  f"group {g} {path}")
        assert padding_untouched(d)


def test_far_rows():
    """Operands and outputs whose rows lie past 32-bit offsets."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(4)
    M, pitch, K, N = 40000, 60000, 64, 72
    x = torch.zeros(M, pitch, dtype=torch.bfloat16, device=DEV)[:, :K]
    y = torch.zeros(M, pitch, dtype=torch.bfloat16, device=DEV)[:, :N]
    x.copy_(torch.randn(M, K, generator=gen).to(torch.bfloat16))
    w = randn(gen, 3, N, K, dtype="bf16", scale=0.1)
    sizes = [20000, 19000, 1000]
    s = torch.cuda.current_stream()
    dgt.gemm_linear(M, N, K, "bf16", 0, 1, x, pitch, w, K, None, "none", None, 0, y, pitch, "bf16", stream=s)
    wy, _, ty, _ = linear_want(x, w[0].T, None, None, "none", "bf16", "bf16")
    close(y, wy, ty, dgt.gemm_last_path())
    dgt.gemm_grouped(3, M, N, K, "bf16", 1, offsets_of(sizes), x, pitch, w, K, N * K, None, "silu", None, 0, y,
                     pitch, "bf16", stream=s)
    wy, _, ty, _ = linear_want(x[39000:], w[2].T, None, None, "silu", "bf16", "bf16")
    close(y[39000:], wy, ty, dgt.gemm_last_path())
    dw = out(3, N, K, dtype="f32")
    dgt.gemm_grouped_grad_weight(3, M, N, K, "bf16", offsets_of(sizes), y, pitch, x, pitch, dw, K, N * K, "f32",
                                 stream=s)
    a, b = y[39000:].double(), x[39000:].double()
    close(dw[2], a.T @ b, sum_tol(1000, a.abs().T @ b.abs()) + tiny("f32"), dgt.gemm_last_path())


def test_other_stream_and_repeat():
    """A call on a side stream after its inputs' work; the same call twice gives the same bits."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(6)
    x, w = randn(gen, 200, 520, dtype="f16"), randn(gen, 264, 520, dtype="f16")
    side = torch.cuda.Stream()
    x2 = x * 2
    side.wait_stream(torch.cuda.current_stream())
    ys = []
    for _ in range(2):
        y = torch.empty(200, 264, dtype=torch.float16, device=DEV)
        with torch.cuda.stream(side):
            dgt.gemm_linear(200, 264, 520, "f16", 0, 1, x2, 520, w, 520, None, "gelu", None, 0, y, 264, "f16",
                            stream=side)
        ys.append(y)
    torch.cuda.synchronize()
    wy, _, ty, _ = linear_want(x2, w.T, None, None, "gelu", "f16", "f16")
    close(ys[0], wy, ty)
    assert torch.equal(ys[0], ys[1])


