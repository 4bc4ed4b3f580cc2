"""The layer operators that move rows and ids, against plain definitions in 64 bits: activation
and bias gradients, tokens sorted by expert, rows sent out and joined, and their gradients."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import (ACTS, ACT_STEPS, DEV, U32, act64, close, half_step, ld, offsets_of, out,
                           padding_untouched, randn, slope64, tiny)

pytestmark = pytest.mark.gpu


def workspace(nbytes):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)


def act_grad(gen, M, N, dtype, act, sizes=None, spare=0, pad=0, inplace=False, want=("dz", "db")):
    import dense_gemm_tile_amd as dgt
    G = 1 if sizes is None else len(sizes)
    used = M if sizes is None else sum(sizes)
    M = used + spare if sizes is not None else M
    say(f"act_grad {M}x{N} {dtype} {act} groups={sizes and sizes[:8]} pad={pad} inplace={inplace}")
    dy, z = randn(gen, M, N, dtype=dtype, pad=pad), randn(gen, M, N, dtype=dtype, pad=pad, scale=2)
    g = dy.double() * (slope64(z.double(), act))
    tol = ACT_STEPS * U32 * (dy.double().abs() * (1 + z.double().abs()))
    dz = (dy if inplace else out(M, N, dtype=dtype, pad=pad)) if "dz" in want else None
    db = out(G, N) if "db" in want else None
    size = dgt.gemm_act_grad_workspace(G, M, N)
    off = None if sizes is None else offsets_of(sizes)
    dgt.gemm_act_grad(G, M, N, dtype, act, off, dy, ld(dy), z, ld(z), dz, ld(dz), db, workspace(size), size,
                      stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    if dz is not None:
        close(dz[:used], g[:used], tol[:used] * 1.01 + half_step(dtype) * g[:used].abs() + tiny(dtype), "dZ")
        if not inplace:
            assert torch.isnan(dz[used:]).all()
        assert padding_untouched(dz)
    if db is not None:
        lo = 0
        for i, n in enumerate(sizes or [M]):
            s = slice(lo, lo + n)
            lo += n
            close(db[i], g[s].sum(0), (tol[s] + (n + 2) * U32 * g[s].abs()).sum(0) + tiny("f32"), f"db {i}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_act_grad(dtype, act):
    need_gpu()
    gen = torch.Generator().manual_seed(1)
    for M, N in ((1, 1), (1, 8), (31, 7), (32, 512), (33, 520), (100, 1000), (1000, 64), (4097, 136)):
        act_grad(gen, M, N, dtype, act)
    act_grad(gen, 70, 64, dtype, act, pad=8)
    act_grad(gen, 70, 64, dtype, act, pad=3)
    act_grad(gen, 70, 64, dtype, act, inplace=True)
    act_grad(gen, 70, 64, dtype, act, want=("dz",))
    act_grad(gen, 70, 64, dtype, act, want=("db",))


@pytest.mark.parametrize("sizes", [[0], [1], [5, 0, 3], [0, 0, 64, 0], [32, 32, 1, 31, 200], [17] * 9,
                                   [1, 0, 0, 2] * 20, [256, 255, 257, 0, 3], [0] * 5])
def test_act_grad_groups(sizes):
    need_gpu()
    gen = torch.Generator().manual_seed(2)
    for N, spare in ((72, 0), (520, 40), (33, 1)):
        act_grad(gen, 0, N, "bf16", "silu", sizes=sizes, spare=spare)
        act_grad(gen, 0, N, "f16", "none", sizes=sizes, spare=spare, want=("db",))


def test_act_grad_row_ends_and_starts():
    """Every number of columns past the last whole piece, at pitches that put rows at any 2-byte
    address; padding stays as it was."""
    need_gpu()
    gen = torch.Generator().manual_seed(3)
    for i in range(16):
        for base in (0, 512):
            N = base + i + 1
            act_grad(gen, 9, N, ("f16", "bf16")[i % 2], ACTS[i % 5], pad=i % 4)
            act_grad(gen, 9, N, ("bf16", "f16")[i % 2], ACTS[(i + 1) % 5], pad=(i + 1) % 3, inplace=True)


@pytest.mark.parametrize("M,N", [(128, 1030), (300, 1030), (520, 4099), (5000, 2050), (20000, 2056)])
def test_act_grad_rows_of_a_wave(M, N):
    """Sizes at which a wave takes 1, 2, 4 and more rows, with groups that end inside its rows."""
    need_gpu()
    gen = torch.Generator().manual_seed(4)
    act_grad(gen, M, N, "bf16", "gelu", pad=1)
    act_grad(gen, 0, N, "f16", "silu", sizes=[M // 3, 0, 1, M // 2 - 1, 5], spare=7, inplace=True)


def test_act_grad_no_rows_gives_zero_sums():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    db = out(1, 40)
    size = dgt.gemm_act_grad_workspace(1, 0, 40)
    dgt.gemm_act_grad(1, 0, 40, "bf16", "gelu", None, None, 40, None, 40, None, 0, db, workspace(size), size)
    torch.cuda.synchronize()
    assert torch.equal(db, torch.zeros_like(db))


@pytest.mark.parametrize("act", ACTS)
def test_act_grad_is_the_slope(act):
    """Against differences of the activation, and at numbers where parts of the formula overflow."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    z = torch.cat([torch.linspace(-12, 12, 2001), torch.tensor([-3e38, -1e20, -100.0, 100.0, 1e20, 3e38])])
    z = z.to(torch.bfloat16).to(DEV)[None]
    dy, dz = torch.ones_like(z), torch.empty_like(z)
    dgt.gemm_act_grad(1, 1, z.shape[1], "bf16", act, None, dy, z.shape[1], z, z.shape[1], dz, z.shape[1], None,
                      None, 0, stream=torch.cuda.current_stream())
    z64, got = z.double(), dz.double()
    h = 1e-4
    d = (act64(z64 + h, act) - act64(z64 - h, act)) / (2 * h)
    far = z64.abs() > 50
    d = torch.where(far & (act != "none"), (z64 > 0).double(), d)
    if act == "none":
        d = torch.ones_like(d)
    kink = (z64.abs() <= h) if act == "relu" else torch.zeros_like(far)
    # half a bf16 step, the difference's own error (h^2/6 of the third derivative, below 1), and
    # float32 arithmetic
    tol = half_step("bf16") * d.abs() + 1e-7 + ACT_STEPS * U32 * (1 + z64.abs().clamp(max=50))
    close(torch.where(kink, d, got), d, tol, act)


def route_want(ids, E):
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(E + 1)]
    for i, e in enumerate(flat):
        lists[e if 0 <= e < E else E].append(i)
    order, offsets, slot = [], [0], [-1] * len(flat)
    for e in range(E):
        for i in lists[e]:
            slot[i] = len(order)
            order.append(i)
        offsets.append(len(order))
    return offsets, order + lists[E], slot


def route(ids, E):
    import dense_gemm_tile_amd as dgt
    T, top = ids.shape
    ids = ids.to(DEV, torch.int32)
    offsets = torch.full((E + 1,), -7, dtype=torch.int32, device=DEV)
    order, slot = (torch.full((T * top,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    size = dgt.gemm_route_workspace(T, top, E)
    dgt.gemm_route(T, top, E, ids, offsets, order, slot, workspace(size), size,
                   stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return offsets, order, slot


@pytest.mark.parametrize("T,top,E", [(0, 2, 8), (1, 1, 1), (1, 1, 2), (7, 2, 4), (63, 1, 64), (65, 8, 128), (1000, 4, 7),
                                     (4096, 4, 256), (4097, 4, 60), (16384, 8, 128), (5000, 6, 1023), (300, 5, 1024),
                                     (9000, 2, 1024), (300000, 8, 32), (40, 3, 0)])
def test_route(T, top, E):
    need_gpu()
    say(f"route T={T} top={top} E={E}")
    gen = torch.Generator().manual_seed(T + E)
    for low, high in ((0, max(E, 1)), (-1, E + 2)):
        ids = torch.randint(low, high, (T, top), generator=gen)
        offsets, order, slot = route(ids, E)
        wo, wr, ws = route_want(ids, E)
        assert offsets.tolist() == wo
        assert order.tolist() == wr
        assert slot.tolist() == ws


def test_route_odd_ids():
    need_gpu()
    for fill in (-1, 5, 2 ** 31 - 1, -2 ** 31, 3):
        ids = torch.full((700, 3), fill, dtype=torch.int64)
        offsets, order, slot = route(ids, 4)
        wo, wr, ws = route_want(ids, 4)
        assert (offsets.tolist(), order.tolist(), slot.tolist()) == (wo, wr, ws)


def slots(gen, T, top, drop):
    """A random placement of the kept choices; -1, and one number past the rows, for the others."""
    n = T * top
    slot = torch.randperm(n, generator=gen).to(torch.int32)
    slot[torch.rand(n, generator=gen) < drop] = -1
    if drop:
        slot[0] = n + 3  # named by no row: skipped like a dropped one
    return slot.reshape(T, top).to(DEV)


ROWS = [(1, 1, 8), (1, 4, 2048), (3, 2, 7), (5, 3, 66), (33, 8, 520), (130, 4, 1032), (17, 5, 4100), (64, 1, 3)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_dispatch_and_its_gradient(dtype, pad):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(3)
    s = torch.cuda.current_stream()
    for T, top, H in ROWS:
        for drop in (0.0, 0.3, 1.0):
            say(f"dispatch {T}x{top}x{H} {dtype} pad={pad} drop={drop}")
            slot, n = slots(gen, T, top, drop), T * top
            kept = (slot >= 0) & (slot < n)
            x, xs = randn(gen, T, H, dtype=dtype, pad=pad), out(n, H, dtype=dtype, pad=pad)
            dgt.gemm_dispatch(T, top, H, dtype, x, ld(x), slot, xs, ld(xs), stream=s)
            want = torch.full((n, H), float("nan"), dtype=torch.float64, device=DEV)
            want[slot[kept].long()] = x.double()[torch.nonzero(kept)[:, 0]]
            close(xs, want, torch.zeros_like(want), "Xs")
            assert padding_untouched(xs)
            dxs, dx = randn(gen, n, H, dtype=dtype, pad=pad), out(T, H, dtype=dtype, pad=pad)
            dgt.gemm_combine(T, top, H, dtype, dxs, ld(dxs), slot, None, None, 0, dx, ld(dx), stream=s)
            rows = dxs.double()[slot.clamp(0, n - 1).long()] * kept[:, :, None]
            want, mag = rows.sum(1), rows.abs().sum(1)
            close(dx, want, top * U32 * mag * 1.01 + half_step(dtype) * want.abs() + tiny(dtype), "dX")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_combine_and_its_gradient(dtype, pad):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(4)
    s = torch.cuda.current_stream()
    for i, (T, top, H) in enumerate(ROWS):
        for drop in (0.0, 0.3, 1.0):
            say(f"combine {T}x{top}x{H} {dtype} pad={pad} drop={drop}")
            slot, n = slots(gen, T, top, drop), T * top
            kept = (slot >= 0) & (slot < n)
            at = slot.clamp(0, n - 1).long()
            ys, w = randn(gen, n, H, dtype=dtype, pad=pad), randn(gen, T, top)
            r = randn(gen, T, H, dtype=dtype, pad=pad) if i % 2 else None
            y = out(T, H, dtype=dtype, pad=pad)
            if i % 4 == 1:
                y.copy_(r)
            rin = y if i % 4 == 1 else r
            dgt.gemm_combine(T, top, H, dtype, ys, ld(ys), slot, w, rin, ld(rin), y, ld(y), stream=s)
            rows = ys.double()[at] * (w.double() * kept)[:, :, None]
            want, mag = rows.sum(1), rows.abs().sum(1)
            if r is not None:
                want, mag = want + r.double(), mag + r.double().abs()
            close(y, want, (top + 2) * U32 * mag * 1.01 + half_step(dtype) * want.abs() + tiny(dtype), "Y")
            assert padding_untouched(y)
            dy, dys, dw = randn(gen, T, H, dtype=dtype, pad=pad), out(n, H, dtype=dtype, pad=pad), out(T, top)
            dgt.gemm_combine_grad(T, top, H, dtype, dy, ld(dy), ys, ld(ys), slot, w, dys, ld(dys), dw, stream=s)
            prod = dy.double()[:, None, :] * ys.double()[at] * kept[:, :, None]
            close(dw, prod.sum(-1), (H + 2) * U32 * prod.abs().sum(-1) + tiny("f32"), "dweights")
            want = torch.full((n, H), float("nan"), dtype=torch.float64, device=DEV)
            g = w.double()[:, :, None] * dy.double()[:, None, :]
            want[slot[kept].long()] = g[kept]
            close(dys, want, torch.nan_to_num((U32 + half_step(dtype)) * 1.01 * want.abs()) + tiny(dtype), "dYs")
            # one output at a time, and the rows' gradient in place of the rows
            dw2, ys2 = out(T, top), out(n, H, dtype=dtype, pad=pad)
            ys2.copy_(ys)
            dgt.gemm_combine_grad(T, top, H, dtype, dy, ld(dy), ys2, ld(ys2), slot, w, None, 0, dw2, stream=s)
            assert torch.equal(dw2, dw)
            dgt.gemm_combine_grad(T, top, H, dtype, dy, ld(dy), ys2, ld(ys2), slot, w, ys2, ld(ys2), dw2, stream=s)
            assert torch.equal(dw2, dw)
            assert torch.equal(ys2[slot[kept].long()], dys[slot[kept].long()])


def test_combine_reads_no_dropped_row():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    ys = torch.full((4, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    ys[2] = 3
    slot = torch.tensor([[2, -1], [-1, -1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, float("nan")], [float("nan"), 1.0]], device=DEV)
    y = out(2, 64, dtype="bf16")
    dgt.gemm_combine(2, 2, 64, "bf16", ys, 64, slot, w, None, 0, y, 64, stream=torch.cuda.current_stream())
    assert torch.equal(y[0], torch.full_like(y[0], 1.5)) and torch.equal(y[1], torch.zeros_like(y[1]))


