"""The gate without a bias: experts by their logits, whatever else a token holds; choices that are dropped beside a
NaN."""
import math

import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, DT
from test_layer_gate_gpu import gate, scores64

pytestmark = pytest.mark.gpu


def falling(key, masked):
    keep = [e for e in range(len(key)) if not masked[e]]
    return sorted(keep, key=lambda e: (1, 0.0, e) if math.isnan(key[e]) else (0, -key[e], e))


def choose_by_logits(L, score, groups, top_groups, group_top, top):
    """Ids without a bias (-1: dropped). Experts are compared by their logits, the NaN scores last; groups by
    their largest expert, or by the sum of their two largest scores in 64 bits."""
    L = L.double().cpu()
    s, size, found = scores64(L, score), L.shape[1] // groups, []
    for t in range(L.shape[0]):
        score_t = s[t].tolist()
        key = [math.nan if math.isnan(x) else l for x, l in zip(score_t, L[t].tolist())]
        masked = [l == -math.inf for l in L[t].tolist()]
        if groups > 1:
            rank, empty = [], []
            for g in range(groups):
                best = [e for e in falling(key, masked) if g * size <= e < (g + 1) * size][:group_top]
                rank.append(math.nan if not best else key[best[0]] if group_top == 1 else sum(score_t[e] for e in best))
                empty.append(not best)
            kept = set((falling(rank, empty) + [g for g in range(groups) if empty[g]])[:top_groups])
            masked = [m or e // size not in kept for e, m in enumerate(masked)]
        ids = falling(key, masked)[:top]
        found.append(ids + [-1] * (top - len(ids)))
    return torch.tensor(found, dtype=torch.int32)


def same_choice(L, dtype, score, groups, top_groups, group_top, top, renorm=True):
    say(f"order {tuple(L.shape)} {dtype} {score} {groups},{top_groups},{group_top}")
    L = L.to(DEV, DT[dtype])
    ids, w = gate(L, dtype, score, None, groups, top_groups, group_top, top, renorm, 1.0)
    want = choose_by_logits(L, score, groups, top_groups, group_top, top)
    assert torch.equal(ids.cpu(), want), (ids.cpu(), want)
    return ids, w


FORMS = [(8, 1, 1, 1), (64, 8, 4, 1), (130, 65, 5, 1), (130, 65, 5, 2), (64, 8, 4, 2), (300, 1, 1, 1), (1000, 1, 1, 1),
         (700, 7, 3, 1)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("E,groups,top_groups,group_top", FORMS)
def test_scores_that_64_bits_do_not_tell_apart(dtype, E, groups, top_groups, group_top):
    """Sigmoid scores of 1 and softmax scores of 0: the larger logit first, also where another logit of the token is
    NaN or next to a third one, and in forms that are in 64 bits throughout."""
    need_gpu()
    gen = torch.Generator().manual_seed(E)
    high = 40.0 + 10 * torch.rand(30, E, generator=gen)  # sigmoid: 1 in 64 bits
    for extra in ("none", "nan", "close"):
        L = high.clone()
        if extra == "nan":
            L[:, 0] = math.nan
        if extra == "close":  # (one float32 step apart)
            L[:, 1], L[:, 3] = 50.5, 50.5 + 2.0 ** -18
        same_choice(L, dtype, "sigmoid", groups, top_groups, group_top, 5)
    low = -800.0 - 100 * torch.rand(30, E, generator=gen)  # softmax beside a 0: 0 in 64 bits
    low[:, 2] = 0
    same_choice(low, dtype, "softmax", groups, top_groups, group_top, 5, renorm=False)
    low[:, 1], low[:, 3] = -750.0, -750.0 - 2.0 ** -14
    same_choice(low, dtype, "softmax", groups, top_groups, group_top, 5)
    low[:, 1] = math.nan  # all scores are NaN
    same_choice(low, dtype, "softmax", groups, top_groups, group_top, 5)
    lowest = torch.full((30, E), torch.finfo(DT[dtype]).min)
    lowest[:, 5] = 1.0
    lowest[:, 7] = -1.0
    for score in ("softmax", "sigmoid"):
        same_choice(lowest, dtype, score, groups, top_groups, group_top, 5)


def test_a_token_alone_and_beside_others():
    """The same two experts in the same order, whatever the token's other logits make of it."""
    need_gpu()
    for hi, lo, score in ((50.0, 40.0, "sigmoid"), (-800.0, -900.0, "softmax")):
        base = [lo, hi] + [-1000.0] * 6
        if score == "softmax":
            base[2] = 0.0
        for change in ((), (3, math.nan), (3, hi * (1 + 2.0 ** -23))):
            if change and score == "softmax" and math.isnan(change[1]):
                continue
            row = list(base)
            if change:
                row[change[0]] = change[1]
            ids, _ = gate(torch.tensor([row], device=DEV), "f32", score, None, 1, 1, 1, 5, False, 1.0)
            ids = ids[0].tolist()
            assert ids.index(1) < ids.index(0), (score, change, ids)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_dropped_choices_beside_nan(score, renorm):
    """A choice without an expert has the weight 0, whatever the others' weights are."""
    need_gpu()
    for E, groups in ((8, 1), (64, 8), (130, 65)):
        L = torch.full((3, E), -math.inf)
        L[:, 1], L[1:, 0] = math.nan, 2.0
        ids, w = gate(L.to(DEV), "f32", score, None, groups, groups, 1, 4, renorm, 1.0)
        assert ids.tolist() == [[1, -1, -1, -1], [0, 1, -1, -1], [0, 1, -1, -1]]
        assert torch.isnan(w[0, 0]) and torch.isnan(w[1:, 1]).all()
        assert (w[0, 1:] == 0).all() and (w[1:, 2:] == 0).all()
