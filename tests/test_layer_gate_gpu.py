"""The gate: chosen experts, weights and the logits' gradient against plain definitions in 64 bits."""
import math

import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, U32, close, half_step, ld, out, padding_untouched, randn, tiny

pytestmark = pytest.mark.gpu


def scores64(logits, score):
    if score == "sigmoid":
        return torch.sigmoid(logits)
    # (A row without experts has no scores: its weights and its gradient are 0.)
    empty = torch.isneginf(logits).all(1, keepdim=True)
    s = torch.softmax(torch.where(empty, torch.zeros_like(logits), logits), 1)
    return torch.where(empty, torch.zeros_like(s), s)


def order(key, masked):
    """Indices by falling key: masked ones out, NaN last, equal ones by rising index."""
    keep = [e for e in range(len(key)) if not masked[e]]
    return sorted(keep, key=lambda e: (1, 0.0, e) if math.isnan(key[e]) else (0, -key[e], e))


def choose(logits, score, bias, groups, top_groups, group_top, top):
    """Ids (-1: dropped) in 64 bits, token by token."""
    L = logits.double().cpu()
    s = scores64(L, score)
    b = torch.zeros(L.shape[1], dtype=torch.float64) if bias is None else bias.double().cpu()
    size = L.shape[1] // groups
    found = []
    for t in range(L.shape[0]):
        key = (s[t] + b).tolist()
        masked = [math.isinf(x) and x < 0 or math.isinf(y) and y < 0 for x, y in zip(L[t].tolist(), b.tolist())]
        if groups > 1:
            rank, empty = [], []
            for g in range(groups):
                best = [e for e in order(key, masked) if g * size <= e < (g + 1) * size][:group_top]
                rank.append(sum(key[e] for e in best))
                empty.append(not best)
            by = order(rank, empty) + [g for g in range(groups) if empty[g]]
            kept = set(by[:top_groups])
            masked = [m or e // size not in kept for e, m in enumerate(masked)]
        ids = order(key, masked)[:top]
        found.append(ids + [-1] * (top - len(ids)))
    return torch.tensor(found, dtype=torch.int32)


def weights64(logits, ids, score, renorm, scale):
    """The chosen scores as weights, differentiable in the logits; ids -1 give 0."""
    s = scores64(logits, score)
    kept = ids >= 0
    w = torch.where(kept, s.gather(1, ids.clamp(min=0).long()), torch.zeros((), dtype=s.dtype, device=s.device))
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, w, w / torch.where(total == 0, torch.ones_like(total), total))
    return w * scale


def gate(L, dtype, score, bias, groups, top_groups, group_top, top, renorm, scale):
    import dense_gemm_tile_amd as dgt
    T, E = L.shape
    ids = torch.full((T, top), -9, dtype=torch.int32, device=DEV)
    w = out(T, top)
    dgt.gemm_gate(T, E, top, dtype, L, ld(L), score, bias, groups, top_groups, group_top, renorm, scale, ids, w,
                  stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    return ids, w


def weight_tol(E, top, want):
    """One exponential, a sum over the experts (a lane adds E / 64 of them, then the lanes are joined)
    and over the choices, two divisions and a factor: a few half steps each."""
    return (E / 64 + top + 32) * U32 * want.abs() + tiny("f32")


def check(gen, T, E, top, dtype="f32", score="softmax", bias=False, groups=1, top_groups=1, group_top=1, renorm=True,
          scale=1.0, pad=0, size=1.5, logits=None):
    import dense_gemm_tile_amd as dgt
    say(f"gate {T}x{E} top={top} {dtype} {score} bias={bias} groups={groups},{top_groups},{group_top} {renorm} pad={pad}")
    L = randn(gen, T, E, dtype=dtype, pad=pad, scale=size) if logits is None else logits
    b = 0.2 * randn(gen, 1, E)[0] if bias is True else bias if bias is not False else None
    ids, w = gate(L, dtype, score, b, groups, top_groups, group_top, top, renorm, scale)
    want = choose(L, score, b, groups, top_groups, group_top, top)
    assert torch.equal(ids.cpu(), want), (ids.cpu() != want).nonzero()[:4]
    L64 = L.double().detach().requires_grad_(True)
    w64 = weights64(L64, ids, score, renorm, scale)
    close(w, w64.detach(), weight_tol(E, top, w64.detach()), "weights")
    dw = randn(gen, T, top)
    dw[ids < 0] = float("nan")  # not read
    dl = out(T, E, dtype=dtype, pad=pad)
    dgt.gemm_gate_grad(T, E, top, dtype, L, ld(L), score, renorm, scale, ids, dw, dl, ld(dl),
                       stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.nan_to_num(dw.double())
    want = torch.autograd.grad((w64 * g).sum(), L64)[0]
    # The derivative of each weight by its own score, at most, and of every score by its sum.
    wv = w64.detach()
    size = (wv * g).abs().sum(1, keepdim=True)
    own = torch.zeros_like(want).scatter_add(1, ids.clamp(min=0).long(), (wv * g).abs() * (ids >= 0))
    s = scores64(L.double(), score)
    share = torch.zeros_like(s).scatter_add(1, ids.clamp(min=0).long(), wv / abs(scale)) if renorm else s
    tol = (E / 64 + top + 64) * U32 * (2 * own + 2 * share * size)
    # The reference rounds as well. An expert that is not chosen has the exact gradient 0 under
    # renormalised softmax weights, where the reference, through the softmax of all of them, has
    # s * (a sum of `top` terms that cancel): each term, and each of the sum's partial results, is off by
    # half a step of 64 bits of at most `size`, after about ten operations of its own.
    tol = tol + (top + 32) * 2.0 ** -53 * s * size / abs(scale) * max(1.0, abs(scale))
    close(dl, want, tol + half_step(dtype) * want.abs() + tiny(dtype), "dL")
    assert padding_untouched(dl)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_and_its_gradient(dtype, score):
    need_gpu()
    gen = torch.Generator().manual_seed(1)
    for T, E, top in ((1, 1, 1), (1, 2, 1), (5, 8, 2), (33, 64, 4), (7, 65, 8), (9, 128, 6), (40, 200, 8), (6, 256, 8),
                      (5, 300, 64), (4, 512, 8), (3, 1000, 10), (2, 1024, 64), (3, 64, 64)):
        for renorm in (False, True):
            check(gen, T, E, top, dtype, score, renorm=renorm)
            check(gen, T, E, top, dtype, score, bias=True, renorm=renorm, scale=2.5, pad=3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups(score, group_top):
    need_gpu()
    gen = torch.Generator().manual_seed(2)
    for T, E, groups, top_groups, top in ((9, 8, 2, 1, 2), (20, 64, 8, 4, 6), (5, 256, 8, 4, 8), (6, 96, 3, 2, 5),
                                          (4, 512, 128, 100, 8), (3, 1024, 512, 60, 9), (3, 700, 7, 7, 8), (3, 130, 65, 3, 4)):
        check(gen, T, E, top, "f32", score, bias=True, groups=groups, top_groups=top_groups, group_top=group_top)
        check(gen, T, E, top, "bf16", score, groups=groups, top_groups=top_groups, group_top=group_top, renorm=False)
    check(gen, 5, 12, 2, groups=12, top_groups=3)  # groups of one
    for E in (1, 8, 200):  # a single group: no ranks
        check(gen, 5, E, 1, "f32", score, group_top=group_top)
        check(gen, 5, E, 1, "bf16", score, bias=True, group_top=group_top)


def test_equal_scores_take_the_lowest_number():
    need_gpu()
    gen = torch.Generator().manual_seed(3)
    for E, top in ((8, 3), (64, 8), (200, 64), (1024, 16)):
        for fill in (0.0, -60000.0, 3.0):
            check(gen, 4, E, top, "f16", logits=torch.full((4, E), fill, dtype=torch.float16, device=DEV))
        L = torch.randint(0, 3, (50, E), generator=gen).to(DEV, torch.bfloat16)
        check(gen, 50, E, top, "bf16", logits=L)
        check(gen, 50, E, top, "bf16", "sigmoid", logits=L, bias=torch.full((E,), 0.5, device=DEV))
        check(gen, 50, E, top, "bf16", logits=L, groups=4, top_groups=2, group_top=2)


def test_scores_that_differ_in_64_bits_alone():
    """Keys closer than float32 tells apart are still ordered: biases that all but cancel the scores'
    differences, and logits of one float32 step."""
    need_gpu()
    gen = torch.Generator().manual_seed(4)
    for score in ("softmax", "sigmoid"):
        L = torch.randn(200, 64, generator=gen)
        L[:, 1:] = L[:, :1] + torch.randint(-3, 4, (200, 63), generator=gen) * 2.0 ** -22
        check(gen, 200, 64, 8, "f32", score, logits=L.to(DEV))
        check(gen, 200, 64, 8, "f32", score, logits=L.to(DEV), groups=8, top_groups=3, group_top=2)
        L = torch.randn(1, 64, generator=gen).expand(200, 64).contiguous()
        bias = (0.75 - scores64(L.double(), score)[0]).float()  # every key is 0.75 to float32
        check(gen, 200, 64, 8, "f32", score, logits=L.to(DEV), bias=bias.to(DEV))
        check(gen, 200, 64, 8, "f32", score, logits=L.to(DEV), bias=bias.to(DEV), groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_few_close_scores(score):
    """Two, three or more keys in a row that float32 does not tell apart, among and beyond the choices, in one
    lane's experts and in several; in all tokens, or in one of many."""
    need_gpu()
    gen = torch.Generator().manual_seed(8)
    for E, top in ((64, 4), (256, 8), (100, 16), (512, 20), (1024, 64)):
        for step, part in ((8.0, 1.0), (2.0, 1.0), (8.0, 0.02)):
            L = torch.randn(150, E, generator=gen)
            near = torch.round(L * step) / step + torch.randint(-2, 3, (150, E), generator=gen) * 2.0 ** -23
            L = torch.where(torch.rand(150, 1, generator=gen) < part, near, L).to(DEV)
            bias = (torch.randint(-2, 3, (E,), generator=gen) * 2.0 ** -24).to(DEV)
            check(gen, 150, E, top, "f32", score, logits=L, bias=bias)
            check(gen, 150, E, top, "f32", score, logits=L, bias=torch.zeros(E, device=DEV), renorm=False)
            check(gen, 150, E, top, "f32", score, logits=L, bias=bias, groups=4, top_groups=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_masked_experts(score, dtype):
    need_gpu()
    gen = torch.Generator().manual_seed(5)
    for E, top in ((8, 4), (64, 8), (300, 6)):
        L = randn(gen, 12, E, dtype=dtype)
        mask = torch.rand(12, E, generator=gen) < 0.6
        mask[0], mask[1], mask[2, : E - 1] = True, False, True
        mask[3, top - 1:] = True
        L[mask.to(DEV)] = -math.inf
        for renorm in (False, True):
            check(gen, 11, E, top, dtype, score, logits=L[1:], renorm=renorm)
            check(gen, 11, E, top, dtype, score, logits=L[1:], renorm=renorm, groups=4, top_groups=2, group_top=2)
        import dense_gemm_tile_amd as dgt
        ids, w = gate(L[:1], dtype, score, None, 1, 1, 1, top, True, 1.0)
        assert (ids == -1).all() and (w == 0).all()
        dl = out(1, E, dtype=dtype)
        dgt.gemm_gate_grad(1, E, top, dtype, L[:1], E, score, True, 1.0, ids, w, dl, E,
                           stream=torch.cuda.current_stream())
        assert torch.equal(dl, torch.zeros_like(dl))
        bias = torch.zeros(E, device=DEV)
        bias[1:] = -math.inf
        ids, w = gate(randn(gen, 3, E, dtype=dtype), dtype, score, bias, 1, 1, 1, top, True, 1.0)
        assert (ids[:, 0] == 0).all() and (ids[:, 1:] == -1).all()
        assert torch.equal(w[:, 0], torch.ones_like(w[:, 0])) and (w[:, 1:] == 0).all()


def test_nan_and_infinity():
    need_gpu()
    L = torch.tensor([[1.0, math.nan, 2.0, 0.0], [1.0, 2.0, 3.0, 4.0], [math.inf, 1.0, 2.0, 0.0]], device=DEV)
    ids, w = gate(L, "f32", "sigmoid", None, 1, 1, 1, 4, False, 1.0)
    assert ids[0].tolist() == [2, 0, 3, 1] and math.isnan(w[0, 3]) and torch.isfinite(w[0, :3]).all()
    assert ids[1].tolist() == [3, 2, 1, 0] and ids[2].tolist()[0] == 0 and w[2, 0] == 1
    ids, w = gate(L, "f32", "softmax", None, 1, 1, 1, 2, True, 1.0)
    assert ids[0].tolist() == [0, 1] and torch.isnan(w[0]).all() and torch.isfinite(w[1]).all()
    assert torch.isnan(w[2]).any()


def test_zero_sums_stay_zero():
    need_gpu()
    L = torch.full((2, 8), -2000.0, device=DEV)  # sigmoid scores of 0 in 64 bits
    ids, w = gate(L, "f32", "sigmoid", None, 1, 1, 1, 2, True, 1.0)
    assert ids.tolist() == [[0, 1], [0, 1]] and (w == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_single_choice_has_the_whole_weight(score):
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(9)
    for T, E in ((300, 64), (40, 500)):
        L, dw = randn(gen, T, E), randn(gen, T, 1)
        ids, w = gate(L, "f32", score, None, 1, 1, 1, 1, True, 2.5)
        assert torch.equal(w, torch.full_like(w, 2.5))
        dl = out(T, E)
        dgt.gemm_gate_grad(T, E, 1, "f32", L, E, score, True, 2.5, ids, dw, dl, E, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(dl, torch.zeros_like(dl))


def test_ids_of_another_program():
    """Ids outside the range are left out; the same one twice counts twice."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(6)
    T, E, top = 6, 20, 4
    ids = torch.tensor([[0, 3, -1, 5], [7, 7, 2, 1], [E, -5, 2 ** 31 - 1, 4], [-1] * 4, [19, 0, 19, 19], [1, 2, 3, 4]],
                       dtype=torch.int32)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            L, dw = randn(gen, T, E), randn(gen, T, top)
            dl = out(T, E)
            dgt.gemm_gate_grad(T, E, top, "f32", L, E, score, renorm, 1.5, ids.to(DEV), dw, dl, E,
                               stream=torch.cuda.current_stream())
            L64 = L.double().requires_grad_(True)
            kept = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, -1)).to(DEV)
            want = torch.autograd.grad((weights64(L64, kept, score, renorm, 1.5) * dw.double()).sum(), L64)[0]
            close(dl, want, torch.full_like(want, 200 * U32 * 10), f"{score} {renorm}")
            same = L.clone()  # in place
            dgt.gemm_gate_grad(T, E, top, "f32", same, E, score, renorm, 1.5, ids.to(DEV), dw, same, E,
                               stream=torch.cuda.current_stream())
            assert torch.equal(same, dl)


def test_gradient_is_the_slope():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(7)
    T, E, top, h = 2, 6, 3, 1e-5
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            L, dw = randn(gen, T, E), randn(gen, T, top)
            ids, _ = gate(L, "f32", score, None, 1, 1, 1, top, renorm, 1.0)
            dl = out(T, E)
            dgt.gemm_gate_grad(T, E, top, "f32", L, E, score, renorm, 1.0, ids, dw, dl, E,
                               stream=torch.cuda.current_stream())
            for i in range(T):
                for j in range(E):
                    e = torch.zeros(T, E, dtype=torch.float64, device=DEV)
                    e[i, j] = h
                    d = sum(k * (weights64(L.double() + k * e, ids, score, renorm, 1.0) * dw.double()).sum()
                            for k in (1, -1)) / (2 * h)
                    assert abs(float(dl[i, j]) - float(d)) < 1e-5
