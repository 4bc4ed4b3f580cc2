"""The gate far from 0: sigmoid scores next to float32's smallest numbers and past 64 bits' smallest, and their
gradient; softmax scores that are 0 in 64 bits."""
import math

import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, DT, U32, close, half_step, out, tiny
from test_layer_gate_gpu import gate

pytestmark = pytest.mark.gpu


def sigmoid_grad(rows, dw, dtype, top):
    """dL of renormalised sigmoid weights of experts 0 .. top - 1 (of them those that have a logit above -infinity),
    and the definition's with what float32 may be off by."""
    import dense_gemm_tile_amd as dgt
    L = torch.tensor(rows, dtype=torch.float64).to(DEV, DT[dtype])
    T, E = L.shape
    g = torch.tensor(dw, dtype=torch.float32, device=DEV)
    ids = torch.arange(top, dtype=torch.int32, device=DEV).expand(T, top).contiguous()
    dl = out(T, E, dtype=dtype)
    dgt.gemm_gate_grad(T, E, top, dtype, L, E, "sigmoid", True, 2.5, ids, g, dl, E, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    # w_j = s_j / S: log s = -log(1 + exp(-l)), and the weights are the softmax of that.
    L64 = L.double().requires_grad_(True)
    w = torch.softmax(torch.nn.functional.logsigmoid(L64[:, :top]), 1)
    want = torch.autograd.grad((2.5 * w * g.double()).sum(), L64)[0]
    # Each share s_j / S: the exponent is a difference of logits (half a step of it, relative to the share), two
    # exponentials, a sum and two divisions, a few half steps each, and the sum over the choices; then
    # the mean, a difference and two products. A share below float32's smallest normal number may count as 0.
    w, g = w.detach(), 2.5 * g.double()
    far = (L64.detach()[:, :top].amax(1, keepdim=True) - L64.detach()[:, :top]).clamp(max=800.0)
    steps = 2 * far + top + 24
    size = g.abs() + (w * g.abs()).sum(1, keepdim=True)
    tol = torch.zeros_like(want)
    tol[:, :top] = U32 * w * (steps * size + (w * g.abs() * steps).sum(1, keepdim=True))
    tol[:, :top] += 2.0 ** -126 * (size + g.abs().sum(1, keepdim=True))
    return dl, want, tol + half_step(dtype) * want.abs() + tiny(dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_gradient_of_small_sigmoid_scores(dtype):
    """Scores whose reciprocal, or themselves, float32 does not hold have weights of ordinary size, and so a
    gradient of ordinary size."""
    need_gpu()
    rest = [-1e4] * 6  # not chosen
    for a, b, c, d in ((-84, -85, 1000, -1000), (-88, -88.25, 10, -10), (-100, -101, 1, 0), (-90, -100, 3, 5), (-87.5, -130, 1, 2),
                       (-300, -302.5, 7, -2), (-600, -600, 1, -1), (-709.5, -709, 1, -1), (-709, -2000, 1, 3), (-60, 2, 1, -1),
                       (-120, 50, 1e4, 2), (-17, -16, 1, 2)):
        say(f"gate_grad {dtype} {a} {b}")
        dl, want, tol = sigmoid_grad([[a, b, *rest], [b, a, *rest]], [[c, d], [c, d]], dtype, 2)
        assert torch.isfinite(dl).all()
        close(dl, want, tol, f"{a} {b}")
    gen = torch.Generator().manual_seed(1)
    for center, spread in ((-30.0, 3.0), (-86.0, 2.0), (-95.0, 2.0), (-400.0, 40.0)):
        for E, top in ((8, 3), (64, 8), (300, 6)):
            rows = center + spread * torch.randn(40, E, generator=gen)
            dl, want, tol = sigmoid_grad(rows.tolist(), torch.randn(40, top, generator=gen).tolist(), dtype, top)
            close(dl, want, tol, f"around {center}")


def test_gradient_where_the_scores_sum_is_zero():
    """Chosen scores that are all 0 in 64 bits have the weights 0, whatever the logits, and so no gradient."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    s = torch.cuda.current_stream()
    for fill in (-709.75, -709.8125, -2000.0, -3e38):
        L = torch.full((2, 8), fill, device=DEV)
        L[:, 1] = fill * (1 + 2.0 ** -20)
        ids, w = torch.zeros(2, 2, dtype=torch.int32, device=DEV), out(2, 2)
        dgt.gemm_gate(2, 8, 2, "f32", L, 8, "sigmoid", None, 1, 1, 1, True, 1.0, ids, w, stream=s)
        dl, dw = out(2, 8), torch.tensor([[1.0, -1.0]] * 2, device=DEV)
        dgt.gemm_gate_grad(2, 8, 2, "f32", L, 8, "sigmoid", True, 1.0, ids, dw, dl, 8, stream=s)
        torch.cuda.synchronize()
        if fill > -709.78:
            assert (w > 0.49).all() and (dl[:, 0] > 0.49).all() and (dl[:, 2] < -0.49).all(), (fill, w, dl)
        else:
            assert (w == 0).all() and (dl == 0).all(), (fill, w, dl)


def test_nan_and_infinite_logits_of_the_gradient():
    need_gpu()
    import dense_gemm_tile_amd as dgt
    L = torch.tensor([[math.nan, -100.0, 1.0], [math.inf, -100.0, 1.0], [-math.inf, -100.0, -101.0]], device=DEV)
    ids = torch.tensor([[0, 1], [0, 1], [0, 1]], dtype=torch.int32, device=DEV)
    dl, dw = out(3, 3), torch.tensor([[1.0, 2.0]] * 3, device=DEV)
    dgt.gemm_gate_grad(3, 3, 2, "f32", L, 3, "sigmoid", True, 1.0, ids, dw, dl, 3, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.isnan(dl[0, :2]).all() and dl[0, 2] == 0
    assert dl[1, 0] == 0 and abs(float(dl[1, 1])) < 1e-40 and dl[1, 2] == 0
    assert torch.equal(dl[2], torch.zeros(3, device=DEV))  # a single choice that is left


def test_renormalised_softmax_far_below_the_largest():
    """Choices whose softmax scores are 0 in 64 bits still have the weights that their logits give, in every form: a
    bias or the groups can pick them."""
    need_gpu()
    for E, groups, top_groups in ((8, 1, 1), (64, 8, 1), (130, 65, 1)):
        size = E // groups
        L = torch.full((4, E), -3000.0)
        at = torch.arange(2) + (size if groups > 1 else 2)  # chosen by their bias
        L[:, 0] = 0.0
        L[:, at[0]], L[:, at[1]] = -1000.0, -1001.0
        L[1, at[0]] = -3.4e38  # the lowest number beside a number
        L[2, at] = -3.4e38
        L[3, E - 1] = math.nan
        bias = torch.zeros(E)
        bias[at] = torch.tensor([9.0, 8.0])
        ids, w = gate(L.to(DEV), "f32", "softmax", bias.to(DEV), groups, top_groups, 1, 2, True, 2.0)
        assert torch.equal(ids[:3].cpu(), at.to(torch.int32).expand(3, 2)), (E, ids)
        want = 2.0 * torch.softmax(L[:3, at].double(), 1)
        close(w[:3], want.to(DEV), 40 * U32 * want.to(DEV) + 1e-45, "weights")
        assert torch.isnan(w[3]).all()


@pytest.mark.parametrize("base,spread", [(-40, 64), (-88, 15)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_weights_of_small_scores(dtype, base, spread):
    """Scores among float32's subnormal numbers are weights as they are, and so are their gradients."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    T, E, top = 64, 16, 3
    L = (base - spread * torch.rand(T, E, generator=torch.Generator().manual_seed(2))).to(DEV, DT[dtype])
    ids, w = gate(L, dtype, "sigmoid", None, 1, 1, 1, top, False, 1.0)
    L64 = L.double()
    want = torch.sigmoid(L64).gather(1, ids.long())
    assert float(want.min()) > 0 and (base > -88 or float(want.min()) < 2.0 ** -130)
    # An exponential of a number that is held, a sum and a division; among the subnormal numbers the exponential
    # and the quotient are each off by a step of 2^-149 at most.
    close(w, want, 12 * U32 * want + 2 * 2.0 ** -149, "sigmoid")
    dw, dl = torch.full((T, top), 3.0, device=DEV), out(T, E, dtype="f32")
    L32 = L.float()
    dgt.gemm_gate_grad(T, E, top, "f32", L32, E, "sigmoid", False, 1.0, ids, dw, dl, E, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = torch.zeros_like(L64).scatter(1, ids.long(), 3 * want)
    close(dl, want, 16 * U32 * want + 3 * 2 * 2.0 ** -149, "dL")
    # Softmax scores beside a logit of 0, which the difference to it leaves exact here.
    L[:, 0] = 0
    ids, w = gate(L, dtype, "softmax", None, 1, 1, 1, top, False, 1.0)
    want = torch.softmax(L.double(), 1).gather(1, ids.long())
    close(w, want, (E / 16 + 24) * U32 * want + 2 * 2.0 ** -149, "softmax")
