"""Calls of more workgroups than a launch holds along one dimension (2^32 threads): many short rows, and
rows of many columns."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, U32

pytestmark = pytest.mark.gpu


def values(*shape, dtype=torch.bfloat16):
    """Seeded values -4 .. 4 in steps of a half: sums of a few of them and halves of them are exact."""
    gen = torch.Generator(DEV).manual_seed(71)
    return (torch.randint(-8, 9, shape, generator=gen, device=DEV, dtype=torch.int8) * 0.5).to(dtype)


def nan(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def test_many_tokens_of_one_value():
    """2^26 waves and more of dispatch, combine and combine_grad with one wave a token."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    T = 2 ** 26 + 5
    say(f"rows of one value, {T} tokens")
    s = torch.cuda.current_stream()
    slot = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
    slot[5] = -1
    x, xs = values(T, 1), nan(T, 1)
    dgt.gemm_dispatch(T, 1, 1, "bf16", x, 1, slot, xs, 1, stream=s)
    want = x.flip(0)
    want[T - 6] = float("nan")
    assert torch.equal(xs.nan_to_num(99.0), want.nan_to_num(99.0))
    w = torch.full((T,), 0.5, device=DEV)
    y, r = nan(T, 1), values(T, 1)
    dgt.gemm_combine(T, 1, 1, "bf16", xs, 1, slot, w, r, 1, y, 1, stream=s)
    want = 0.5 * x + r
    want[5] = r[5]
    assert torch.equal(y, want)
    dys, dw = nan(T, 1), nan(T, dtype=torch.float32)
    dgt.gemm_combine_grad(T, 1, 1, "bf16", r, 1, xs, 1, slot, w, dys, 1, dw, stream=s)
    want = (0.5 * r).flip(0)
    want[T - 6] = float("nan")
    assert torch.equal(dys.nan_to_num(99.0), want.nan_to_num(99.0))
    want = (x * r)[:, 0].float()
    want[5] = 0
    assert torch.equal(dw, want)


def test_many_tokens_of_longer_rows():
    """2^24 workgroups and more of combine_grad, one a token."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    T, H = 2 ** 24 + 3, 129
    say(f"rows of {H} values, {T} tokens")
    slot = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
    w = torch.full((T,), 0.5, device=DEV)
    dy, ys = values(T, H, dtype=torch.float16), values(T, H, dtype=torch.float16)
    dys, dw = nan(T, H, dtype=torch.float16), nan(T, dtype=torch.float32)
    dgt.gemm_combine_grad(T, 1, H, "f16", dy, H, ys, H, slot, w, dys, H, dw, stream=torch.cuda.current_stream())
    step = 2 ** 21
    for lo in range(0, T, step):
        hi = min(T, lo + step)
        assert torch.equal(dys[T - hi:T - lo], (0.5 * dy[lo:hi]).flip(0)), lo
        prod = dy[lo:hi].double() * ys[T - hi:T - lo].flip(0).double()
        assert ((dw[lo:hi] - prod.sum(1)).abs() <= (H + 2) * U32 * prod.abs().sum(1)).all(), lo


@pytest.mark.parametrize("M,N", [(3, 65535 * 512 + 521), (1, 2 ** 28 + 72)])
def test_act_grad_of_long_rows(M, N):
    """More columns than 65535 blocks of 512, and than a launch of the bias sums holds along x."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    say(f"act_grad {M}x{N}")
    dy, z = values(M, N), values(M, N).flip(1).contiguous()
    dz, db = nan(M, N), nan(1, N, dtype=torch.float32)
    size = dgt.gemm_act_grad_workspace(1, M, N)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    dgt.gemm_act_grad(1, M, N, "bf16", "relu", None, dy, N, z, N, dz, N, db, ws, size,
                      stream=torch.cuda.current_stream())
    want = torch.where(z > 0, dy, torch.zeros_like(dy))
    assert torch.equal(dz, want)
    assert torch.equal(db[0], want.float().sum(0))


def test_a_launch_that_is_too_large_is_an_error(monkeypatch):
    """2^26 and one tiles of gemm() at 64 threads each: nothing is computed, and the call says so."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    M = 2 ** 30 + 16
    say(f"gemm {M}x1x1 on 16x16 tiles")
    monkeypatch.setenv("GEMM_FORCE_TILE", "t16x16x64")
    a, b = torch.ones(M, dtype=torch.bfloat16, device=DEV), torch.ones(1, dtype=torch.bfloat16, device=DEV)
    d = nan(M, dtype=torch.float32)
    s = torch.cuda.current_stream()
    with pytest.raises(dgt.GemmError) as e:
        dgt.gemm(M, 1, 1, "bf16", 0, 1, 1.0, 0.0, a, 1, b, 1, None, 1, d, 1, stream=s)
    assert e.value.code == dgt.GEMM_ERR_HIP and "t16x16x64" in dgt.gemm_last_path()
    assert bool(torch.isnan(d).all())
    dgt.gemm(2 ** 30 - 16, 1, 1, "bf16", 0, 1, 1.0, 0.0, a, 1, b, 1, None, 1, d, 1, stream=s)
    assert bool((d[:2 ** 30 - 16] == 1).all()) and bool(torch.isnan(d[2 ** 30 - 16:]).all())
