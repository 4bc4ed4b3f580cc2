"""The layer operators together, as examples/expert_layer.py runs them: values and gradients
against the definition in 64 bits and against differences, a captured graph replayed, and a
training run whose loss falls."""
import importlib.util
import os

import pytest
import torch

from gpu_helpers import need_gpu, say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def definition(p, x, ids, weights):
    """The layer in 64 bits, one expert at a time, in torch."""
    u = torch.nn.functional.gelu(x @ p["w0"].T + p["b0"], approximate="tanh")
    y = x
    for e in range(p["w1"].shape[0]):
        share = (weights * (ids == e)).sum(1, keepdim=True)  # 0 where a token did not choose e
        a = torch.nn.functional.silu(u @ p["w1"][e].T + p["b1"][e])
        y = y + share * (a @ p["w2"][e].T)
    return y


def setup(example, t, h, hidden, experts, top, dtype, drop=0.0):
    gen = torch.Generator().manual_seed(t + h)
    layer = example.ExpertLayer(h, hidden, experts, dtype=dtype)
    for k in ("b0", "b1"):
        layer.master[k] += 0.1 * torch.randn(layer.master[k].shape, generator=gen).cuda()
    layer.cast()
    x = torch.randn(t, h, generator=gen).cuda().to(dtype)
    ids, weights = example.choose(torch.randn(t, experts, generator=gen).cuda(), top)
    if drop:
        ids[(torch.rand(t, top, generator=gen) < drop).cuda()] = -1
    dy = torch.randn(t, h, generator=gen).cuda().to(dtype)
    return layer, x, ids.contiguous(), weights.contiguous(), dy


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


# Every path from an input to an output or gradient passes at most 8 tensors rounded to the
# layer's type; each moves what follows by at most about half a step of it in norm, and the layer's
# own slopes stay near 1.
SHARES = 8 * 2


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,h,hidden,experts,top,drop", [(300, 128, 256, 8, 2, 0.0), (33, 64, 96, 4, 4, 0.3),
                                                         (5, 72, 40, 16, 1, 0.0), (700, 200, 328, 3, 2, 0.1)])
def test_values_and_gradients(example, t, h, hidden, experts, top, drop, dtype):
    need_gpu()
    say(f"expert layer {t}x{h}, {experts} experts of {hidden}, top {top}, drop {drop}, {dtype}")
    layer, x, ids, weights, dy = setup(example, t, h, hidden, experts, top, dtype, drop)
    y, kept = layer.forward(x, ids, weights)
    dx, dweights, grads = layer.backward(dy, kept)
    torch.cuda.synchronize()
    p = {k: v.double().requires_grad_(True) for k, v in layer.w.items()}
    x64, w64 = x.double().requires_grad_(True), weights.double().requires_grad_(True)
    want = definition(p, x64, ids, w64)
    want.backward(dy.double())
    tol = SHARES * torch.finfo(dtype).eps / 2
    assert off(y, want.detach()) <= tol
    assert off(dx, x64.grad) <= tol
    kept_choices = ids >= 0
    assert (dweights[~kept_choices] == 0).all()
    assert off(dweights, w64.grad) <= tol
    for k in p:
        assert off(grads[k], p[k].grad) <= tol, k


def test_gradient_against_differences(example):
    """The loss along a direction in every parameter, from the definition on both sides of it."""
    need_gpu()
    layer, x, ids, weights, dy = setup(example, 200, 64, 128, 4, 2, torch.float16)
    y, kept = layer.forward(x, ids, weights)
    _, _, grads = layer.backward(dy, kept)
    gen = torch.Generator().manual_seed(3)
    x64, w64, step = x.double(), weights.double(), 1e-4
    for k, g in grads.items():
        p = {n: v.double() for n, v in layer.w.items()}
        d = torch.randn(p[k].shape, generator=gen, dtype=torch.float64).cuda() + 3 * g.double() / g.double().norm()
        d /= d.norm()
        losses = []
        for s in (step, -step):
            q = dict(p)
            q[k] = p[k] + s * d
            losses.append((definition(q, x64, ids, w64) * dy.double()).sum())
        slope = float((losses[0] - losses[1]) / (2 * step))
        got = float((g.double() * d).sum())
        # the gradient's own roundings, and the differences' third-order term
        assert abs(got - slope) <= SHARES * 2.0 ** -11 * float(g.double().norm()) + 1e-6 * abs(slope), k


def test_captured_graph_replays(example):
    """Forward and backward captured once and replayed, other work and inputs between the replays:
    every replay equals the eager result of its inputs, bit for bit."""
    need_gpu()
    layer, x, ids, weights, dy = setup(example, 260, 128, 192, 8, 2, torch.bfloat16, 0.1)
    other = [setup(example, 260, 128, 192, 8, 2, torch.bfloat16, d) for d in (0.0, 0.4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.backward(dy, layer.forward(x, ids, weights)[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, kept = layer.forward(x, ids, weights)
        dx, dweights, grads = layer.backward(dy, kept)
    for _, x2, ids2, weights2, dy2 in [other[0], other[1], other[0]]:
        x.copy_(x2), ids.copy_(ids2), weights.copy_(weights2), dy.copy_(dy2)
        graph.replay()
        torch.cuda.synchronize()
        y3, kept3 = layer.forward(x, ids, weights)
        dx3, dweights3, grads3 = layer.backward(dy, kept3)
        assert torch.equal(y, y3) and torch.equal(dx, dx3) and torch.equal(dweights, dweights3)
        for k in grads:
            assert torch.equal(grads[k], grads3[k]), k


def test_training_follows_the_definition(example):
    """Gradient descent beside the same descent in 64 bits. (At this rate the descent itself leaves
    the valley at its twelfth step, in 64 bits too: the steps before it are compared.)"""
    need_gpu()
    layer, x, ids, weights, target = setup(example, 256, 128, 256, 4, 2, torch.bfloat16)
    q = {k: v.double().requires_grad_(True) for k, v in layer.master.items()}
    losses = []
    for _ in range(8):
        y, kept = layer.forward(x, ids, weights)
        error = y.float() - target.float()
        losses.append(float((error * error).mean()))
        _, _, grads = layer.backward((2.0 / 256 * error).to(torch.bfloat16), kept)
        layer.update(grads, 0.1)
        loss = (definition(q, x.double(), ids, weights.double()) - target.double()).square()
        assert abs(losses[-1] - float(loss.detach().mean())) <= SHARES * 2.0 ** -8 * losses[-1]
        (loss.sum() / 256).backward()
        with torch.no_grad():
            for v in q.values():
                v -= 0.1 * v.grad
                v.grad = None
    assert losses[-1] < 0.6 * losses[0], losses
