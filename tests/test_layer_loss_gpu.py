"""The output layer's cross entropy and its gradients against plain definitions in 64 bits."""
import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, U32, close, half_step, ld, out, padding_untouched, randn, sum_tol, tiny

pytestmark = pytest.mark.gpu


def workspace(nbytes):
    # No value of a workspace is meant to be read before the call has written it.
    return torch.full((max(nbytes, 16),), 0xFF, dtype=torch.uint8, device=DEV)


def loss(x, w, labels, dtype, V, keep=True):
    import dense_gemm_tile_amd as dgt
    T, H = x.shape
    found, lse = out(1, T)[0], out(1, T)[0] if keep else None
    size = dgt.gemm_loss_workspace(T, V, H)
    dgt.gemm_loss(T, V, H, dtype, x, ld(x), w, ld(w), labels, found, lse, workspace(size), size,
                  stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return found, lse


def check_loss(x, w, labels, got):
    found, lse = got
    x, w = x.double(), w.double()
    V, H = w.shape
    L, el = x @ w.T, sum_tol(H, x.abs() @ w.abs().T)
    want = torch.logsumexp(L, 1)
    # The logits' errors, those of the exponentials and of their sum (relative: no more than a 256th of
    # them one after the other), and of the logarithm and the addition.
    tol = el.max(1).values + (V / 256 + 64) * U32 + 4 * U32 * (want.abs() + L.abs().max(1).values)
    if lse is not None:
        close(lse, want, tol, "lse")
    has = (labels >= 0) & (labels < V)
    at = labels.clamp(0, V - 1).long()[:, None]
    each = want - L.gather(1, at)[:, 0]
    each, tol = torch.where(has, each, 0 * each), tol + el.gather(1, at)[:, 0] + U32 * each.abs()
    close(found, each, torch.where(has, tol, 0 * tol), "loss")


def check_grad(x, w, labels, lse, dloss, dtype, dx, dw, dw_dtype, before=None):
    x, w = x.double(), w.double()
    V, H = w.shape
    T = x.shape[0]
    L, el = x @ w.T, sum_tol(H, x.abs() @ w.abs().T)
    has = ((labels >= 0) & (labels < V))[:, None]
    p = torch.exp(L - lse.double()[:, None])
    hot = torch.zeros_like(p).scatter_(1, labels.clamp(0, V - 1).long()[:, None], 1.0)
    d = torch.where(has, dloss.double()[:, None], torch.zeros((), dtype=torch.float64, device=DEV))
    G = torch.where(has, (p - hot) * d, 0 * p)
    # exp's argument carries the logit's error and its own rounding; then a difference, a factor and
    # the rounding to 16 bits.
    eg = d.abs() * (p * (el * 1.01 + ((L - lse.double()[:, None]).abs() + 8) * U32) + 2 * U32 * hot) + 2 * U32 * G.abs()
    eg = torch.where(has, eg * 1.01 + half_step(dtype) * G.abs() + tiny(dtype), 0 * p)
    if dx is not None:
        want = G @ w
        tol = eg @ w.abs() + sum_tol(V, (G.abs() + eg) @ w.abs())
        close(dx, want, tol * 1.01 + half_step(dtype) * want.abs() + tiny(dtype), "dX")
    if dw is not None:
        want = G.T @ x
        tol = eg.T @ x.abs() + sum_tol(T, (G.abs() + eg).T @ x.abs())
        if before is not None:
            want = want + before.double()
            tol = tol + U32 * want.abs()
        close(dw, want, tol * 1.01 + half_step(dw_dtype) * want.abs() + tiny(dw_dtype), "dW")


def both(gen, T, V, H, dtype, pad=0, dw_dtype=None, accumulate=False, want=("dx", "dw"), drop=0.2, scale=1.0):
    import dense_gemm_tile_amd as dgt
    o = dw_dtype or dtype
    say(f"loss {T}x{V}x{H} {dtype} pad={pad} dw={o} {accumulate} {want}")
    x, w = randn(gen, T, H, dtype=dtype, pad=pad, scale=scale), randn(gen, V, H, dtype=dtype, pad=pad, scale=H ** -0.5)
    labels = torch.randint(0, V, (T,), generator=gen)
    labels[torch.rand(T, generator=gen) < drop] = -1
    labels[::7] = torch.tensor([V - 1, 0, V, -100, 2 ** 31 - 1])[torch.arange((T + 6) // 7) % 5]
    labels = labels.to(DEV, torch.int32)
    got = loss(x, w, labels, dtype, V)
    check_loss(x, w, labels, got)
    lse = got[1]
    dloss = randn(gen, 1, T)[0] * (64.0 if dtype == "f16" else 1.0)
    dloss[(labels < 0) | (labels >= V)] = float("nan")  # not read
    dx = out(T, H, dtype=dtype, pad=pad) if "dx" in want else None
    dw = (randn(gen, V, H, dtype=o, pad=pad) if accumulate else out(V, H, dtype=o, pad=pad)) if "dw" in want else None
    before = dw.clone() if accumulate else None
    size = dgt.gemm_loss_grad_workspace(T, V, H)
    dgt.gemm_loss_grad(T, V, H, dtype, x, ld(x), w, ld(w), labels, lse, dloss, dx, ld(dx), dw, ld(dw), o, accumulate,
                       workspace(size), size, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    check_grad(x, w, labels, lse, torch.nan_to_num(dloss), dtype, dx, dw, o, before)
    for m in (dx, dw):
        assert m is None or padding_untouched(m)


SIZES = [(1, 1, 1), (1, 2, 8), (3, 7, 5), (17, 100, 64), (5, 1000, 72), (64, 2048, 128), (65, 513, 200), (300, 777, 136),
         (256, 4096, 256), (700, 2050, 64), (1, 5000, 512)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,V,H", SIZES)
def test_loss_and_its_gradients(dtype, T, V, H):
    need_gpu()
    gen = torch.Generator().manual_seed(T + V + H)
    both(gen, T, V, H, dtype)
    both(gen, T, V, H, dtype, pad=3, dw_dtype="f32", accumulate=True, scale=4.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_gradient_at_a_time(dtype):
    need_gpu()
    gen = torch.Generator().manual_seed(3)
    for T, V, H in ((40, 300, 64), (256, 2048, 256)):
        both(gen, T, V, H, dtype, want=("dx",))
        both(gen, T, V, H, dtype, want=("dw",), accumulate=True)
        both(gen, T, V, H, dtype, drop=1.0)


@pytest.mark.parametrize("T,V,H", [(5000, 20000, 64), (9000, 30001, 72), (70000, 1500, 40), (4096, 16896, 128)])
def test_several_pieces(T, V, H):
    """Vocabularies cut into pieces, the last one short, in 64 bits piece by piece."""
    need_gpu()
    both(torch.Generator().manual_seed(T), T, V, H, "bf16", dw_dtype="f32")


@pytest.mark.parametrize("T,V,H,dtype", [(1000, 64 * 256 + 100, 1032, "f16"), (300, 33000, 1024, "bf16"), (200, 65700, 1024, "bf16")])
def test_long_rows_on_many_tiles(T, V, H, dtype):
    """A few tiles more than there are workgroups, dX's sum in parts, rows of more than a slice's multiple."""
    need_gpu()
    both(torch.Generator().manual_seed(T), T, V, H, dtype, dw_dtype="f32")


def test_large_logits():
    """Logits of thousands: exponentials relative to the largest neither overflow nor vanish together."""
    need_gpu()
    gen = torch.Generator().manual_seed(4)
    for T, V, H in ((40, 500, 64), (256, 2048, 128)):
        both(gen, T, V, H, "bf16", scale=1000.0)


def test_no_rows_and_no_width():
    need_gpu()
    import math

    import dense_gemm_tile_amd as dgt
    s = torch.cuda.current_stream()
    dw = out(5, 16)
    dgt.gemm_loss_grad(0, 5, 16, "bf16", None, 16, None, 16, None, None, None, None, 0, dw, 16, "f32", False, None, 0, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(dw, torch.zeros_like(dw))
    labels = torch.tensor([0, 4, -1], dtype=torch.int32, device=DEV)
    found, lse = out(1, 3)[0], out(1, 3)[0]
    size = dgt.gemm_loss_workspace(3, 5, 0)
    dgt.gemm_loss(3, 5, 0, "bf16", None, 1, None, 1, labels, found, lse, workspace(size), size, stream=s)
    close(lse, torch.full((3,), math.log(5.0), dtype=torch.float64, device=DEV), torch.full((3,), 1e-6, device=DEV), "lse")
    assert found[2] == 0 and torch.equal(found[:2], lse[:2])


def test_gradient_is_the_slope():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(5)
    T, V, H, h = 3, 9, 8, 1e-5
    x, w, dloss = randn(gen, T, H, dtype="f16"), randn(gen, V, H, dtype="f16"), randn(gen, 1, T)[0]
    labels = torch.tensor([2, 8, -1], dtype=torch.int32, device=DEV)
    _, lse = loss(x, w, labels, "f16", V)
    dx, dw = out(T, H, dtype="f16"), out(V, H)
    size = dgt.gemm_loss_grad_workspace(T, V, H)
    dgt.gemm_loss_grad(T, V, H, "f16", x, H, w, H, labels, lse, dloss, dx, H, dw, H, "f32", False, workspace(size), size,
                       stream=torch.cuda.current_stream())

    def f(x, w):
        L = x @ w.T
        each = torch.logsumexp(L, 1) - L.gather(1, labels.clamp(min=0).long()[:, None])[:, 0]
        return (each * dloss.double() * (labels >= 0)).sum()
    for m, got in ((0, dx), (1, dw)):
        base = [x.double(), w.double()]
        for i in range(got.shape[0]):
            for j in range(H):
                d = 0.0
                for k in (1, -1):
                    args = [a.clone() for a in base]
                    args[m][i, j] += k * h
                    d += k * float(f(*args)) / (2 * h)
                # G and dX in f16: half a step of each of the V (or T) products, of sizes below 4
                assert abs(float(got[i, j]) - d) < 4 * 10 * 2.0 ** -11, (m, i, j)


def grad(x, w, labels, lse, dloss, dtype, dw_dtype="f32"):
    import dense_gemm_tile_amd as dgt
    (T, H), V = x.shape, w.shape[0]
    dx, dw = out(T, H, dtype=dtype), out(V, H, dtype=dw_dtype)
    size = dgt.gemm_loss_grad_workspace(T, V, H)
    dgt.gemm_loss_grad(T, V, H, dtype, x, ld(x), w, ld(w), labels, lse, dloss, dx, ld(dx), dw, ld(dw), dw_dtype, False,
                       workspace(size), size, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return dx, dw


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,V,H", [(40, 500, 64), (260, 2048, 128), (300, 1000, 72)])
def test_dloss_of_any_size(dtype, T, V, H):
    """A factor 2^k of dloss is the same factor of the gradients, bit for bit: no size of it is rounded away
    (probabilities of 1e-3 and a dloss of 2^-40 would not be numbers of f16, nor 2^40)."""
    need_gpu()
    gen = torch.Generator().manual_seed(7)
    x, w = randn(gen, T, H, dtype=dtype), randn(gen, V, H, dtype=dtype, scale=H ** -0.5)
    labels = torch.randint(0, V, (T,), generator=gen).to(DEV, torch.int32)
    labels[5] = -1
    lse, dloss = loss(x, w, labels, dtype, V)[1], randn(gen, 1, T)[0]
    dx, dw = grad(x, w, labels, lse, dloss, dtype)
    check_grad(x, w, labels, lse, dloss, dtype, dx, dw, "f32")
    for k in (-40, -10, 10, 40):
        got = grad(x, w, labels, lse, dloss * 2.0 ** k, dtype)
        assert torch.equal(got[1], dw * 2.0 ** k), k
        if dtype == "bf16":
            assert torch.equal(got[0], dx * 2.0 ** k), k


@pytest.mark.parametrize("T", [40, 300])
def test_dloss_without_a_value(T):
    """A token's infinite dloss, or its NaN, stays with its row of dX; zeros alone give zeros."""
    need_gpu()
    gen = torch.Generator().manual_seed(8)
    x, w = randn(gen, T, 64, dtype="f16"), randn(gen, 500, 64, dtype="f16", scale=0.125)
    labels = torch.randint(0, 500, (T,), generator=gen).to(DEV, torch.int32)
    lse, dloss = loss(x, w, labels, "f16", 500)[1], torch.full((T,), 0.5, device=DEV)
    want = grad(x, w, labels, lse, dloss, "f16")[0]
    dloss[3], dloss[8], dloss[T - 1] = float("inf"), float("nan"), -float("inf")
    got, bad = grad(x, w, labels, lse, dloss, "f16")[0], [3, 8, T - 1]
    assert not torch.isfinite(got[bad]).any()
    left = torch.ones(T, dtype=torch.bool, device=DEV)
    left[bad] = False
    assert torch.equal(got[left], want[left])
    for m in grad(x, w, labels, lse, 0 * want[:, 0].float(), "f16"):
        assert torch.equal(m, torch.zeros_like(m))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_mean_of_hard_tokens(dtype):
    """Where all tokens weigh the same and are far from their labels, G's largest elements, the labels', are not
    rounded: dW comes out closer than G's rounding to 16 bits would let it, whatever the weight."""
    need_gpu()
    gen = torch.Generator().manual_seed(9)
    T, V, H = 320, 40000, 64
    x, w = randn(gen, T, H, dtype=dtype), randn(gen, V, H, dtype=dtype, scale=0.02)
    labels = torch.randperm(V, generator=gen)[:T].to(DEV, torch.int32)
    lse, weight = loss(x, w, labels, dtype, V)[1], 0.7 / T
    got = grad(x, w, labels, lse, torch.full((T,), weight, device=DEV), dtype)[1][labels.long()].double()
    # Row labels[t]: weight times (p - 1) x[t], and probabilities p below 1e-4 of the other tokens: each
    # product off by half a step at most where it is a p, the label's by the 1e-4 that may round away.
    L = x.double() @ w.double().T
    p = torch.exp(L - lse.double()[:, None])
    assert float(p.max()) < 1e-4
    G = (p[:, labels.long()] - torch.eye(T, dtype=torch.float64, device=DEV)) * weight
    want = G.T @ x.double()
    off = torch.linalg.norm(got - want) / torch.linalg.norm(want)
    print(f"relative error {float(off):.2e}", flush=True)
    assert float(off) < 1.5e-4


def test_products_inside_take_no_named_tile(monkeypatch):
    """GEMM_LAYER_TILE names the kernel of a call's own product, not those of the loss."""
    need_gpu()
    gen = torch.Generator().manual_seed(10)
    x, w = randn(gen, 40, 64, dtype="bf16"), randn(gen, 500, 64, dtype="bf16")
    labels = torch.randint(0, 500, (40,), generator=gen).to(DEV, torch.int32)
    dloss = torch.ones(40, device=DEV)

    def both_calls():
        found, lse = loss(x, w, labels, "bf16", 500)
        return (found, lse, *grad(x, w, labels, lse, dloss, "bf16"))
    want = both_calls()
    for name in ("pp256x256", "no such kernel"):
        monkeypatch.setenv("GEMM_LAYER_TILE", name)
        for a, b in zip(both_calls(), want):
            assert torch.equal(a, b)


def test_runs_repeat():
    need_gpu()
    gen = torch.Generator().manual_seed(6)
    x, w = randn(gen, 300, 128, dtype="bf16"), randn(gen, 3000, 128, dtype="bf16")
    labels = torch.randint(0, 3000, (300,), generator=gen).to(DEV, torch.int32)
    first = loss(x, w, labels, "bf16", 3000)
    for _ in range(3):
        again = loss(x, w, labels, "bf16", 3000)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert torch.equal(loss(x, w, labels, "bf16", 3000, keep=False)[0], first[0])
