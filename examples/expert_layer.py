"""A layer of experts trained and used through the layer operators: tokens pass a linear layer,
are sent to `top` of E experts each (two products with SiLU between them), and come back weighted
onto the residual stream. The forward pass, its gradients and plain gradient descent, on one GPU.

    python examples/expert_layer.py [--steps 30] [--tokens 512]

prints the loss of every fifth step; it has to fall.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_tile_amd as dgt  # noqa: E402

DTYPE = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}


def stream():
    return torch.cuda.current_stream()


def linear(x, w, bias=None, act="none", residual=None, out=None, keep_z=False, trans_a=False, trans_b=True):
    """act(op(x) @ op(w) + bias) + residual, and the sum before act when it is kept."""
    m, k = (x.shape[1], x.shape[0]) if trans_a else x.shape
    n = w.shape[0] if trans_b else w.shape[1]
    y = torch.empty(m, n, dtype=out or x.dtype, device=x.device)
    z = torch.empty(m, n, dtype=x.dtype, device=x.device) if keep_z else None
    dgt.gemm_linear(m, n, k, DTYPE[x.dtype], trans_a, trans_b, x, x.stride(0), w, w.stride(0), bias, act, residual,
                    n, y, n, DTYPE[y.dtype], z, n, stream=stream())
    return (y, z) if keep_z else y


def grouped(x, w, offsets, bias=None, act="none", keep_z=False, trans_b=True):
    """The linear layer with weights w[g] for the rows of group g."""
    groups, rows = w.shape[0], x.shape[0]
    n, k = (w.shape[1], w.shape[2]) if trans_b else (w.shape[2], w.shape[1])
    y = torch.empty(rows, n, dtype=x.dtype, device=x.device)
    z = torch.empty(rows, n, dtype=x.dtype, device=x.device) if keep_z else None
    dgt.gemm_grouped(groups, rows, n, k, DTYPE[x.dtype], trans_b, offsets, x, k, w, w.stride(1), w.stride(0), bias,
                     act, None, 0, y, n, DTYPE[y.dtype], z, n, stream=stream())
    return (y, z) if keep_z else y


def grouped_grad_weight(dy, x, offsets, groups):
    """dy[g]^T @ x[g] of every group, in float32."""
    rows, n, k = dy.shape[0], dy.shape[1], x.shape[1]
    dw = torch.empty(groups, n, k, dtype=torch.float32, device=x.device)
    dgt.gemm_grouped_grad_weight(groups, rows, n, k, DTYPE[x.dtype], offsets, dy, n, x, k, dw, k, n * k, "f32",
                                 stream=stream())
    return dw


def act_grad(dy, z, act, offsets=None, groups=1):
    """dy * act'(z) and its sums over each group's rows, in float32."""
    rows, n = dy.shape
    dz = torch.empty_like(dy)
    db = torch.empty(groups, n, dtype=torch.float32, device=dy.device)
    size = dgt.gemm_act_grad_workspace(groups, rows, n)
    ws = torch.empty(size, dtype=torch.uint8, device=dy.device)
    dgt.gemm_act_grad(groups, rows, n, DTYPE[dy.dtype], act, offsets, dy, n, z, n, dz, n, db, ws, size, stream=stream())
    return dz, db


class ExpertLayer:
    """Weights in 16 bits, float32 masters beside them for the update."""

    def __init__(self, h, hidden, experts, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.experts, self.dtype = experts, dtype
        draw = lambda *s: (torch.randn(*s, generator=gen) * s[-1] ** -0.5).to(device)  # noqa: E731
        self.master = {"w0": draw(h, h), "b0": torch.zeros(h, device=device),
                       "w1": draw(experts, hidden, h), "b1": torch.zeros(experts, hidden, device=device),
                       "w2": draw(experts, h, hidden)}
        self.cast()

    def cast(self):
        self.w = {k: v.to(self.dtype) for k, v in self.master.items()}

    def forward(self, x, ids, weights):
        """x: T x h; ids: T x top int32, -1 for none; weights: T x top float32. Returns y and what
        the backward pass needs."""
        w, (t, h), top, e = self.w, x.shape, ids.shape[1], self.experts
        u, z0 = linear(x, w["w0"], w["b0"], act="gelu", keep_z=True)
        # Where every choice goes, and the rows there.
        offsets = torch.empty(e + 1, dtype=torch.int32, device=x.device)
        order = torch.empty(t * top, dtype=torch.int32, device=x.device)
        slot = torch.empty(t, top, dtype=torch.int32, device=x.device)
        size = dgt.gemm_route_workspace(t, top, e)
        ws = torch.empty(size, dtype=torch.uint8, device=x.device)
        dgt.gemm_route(t, top, e, ids, offsets, order, slot, ws, size, stream=stream())
        us = torch.empty(t * top, h, dtype=x.dtype, device=x.device)
        dgt.gemm_dispatch(t, top, h, DTYPE[x.dtype], u, h, slot, us, h, stream=stream())
        a, z1 = grouped(us, w["w1"], offsets, w["b1"], act="silu", keep_z=True)
        ys = grouped(a, w["w2"], offsets)
        y = torch.empty_like(x)
        dgt.gemm_combine(t, top, h, DTYPE[x.dtype], ys, h, slot, weights, x, h, y, h, stream=stream())
        return y, (x, z0, slot, weights, offsets, us, a, z1, ys)

    def backward(self, dy, kept):
        """Gradients of x, of the choices' weights, and of every parameter."""
        x, z0, slot, weights, offsets, us, a, z1, ys = kept
        (t, h), top, e, w, dt = x.shape, slot.shape[1], self.experts, self.w, DTYPE[x.dtype]
        dys, dweights = torch.empty_like(ys), torch.empty_like(weights)
        dgt.gemm_combine_grad(t, top, h, dt, dy, h, ys, h, slot, weights, dys, h, dweights, stream=stream())
        grads = {"w2": grouped_grad_weight(dys, a, offsets, e)}
        dz1, grads["b1"] = act_grad(grouped(dys, w["w2"], offsets, trans_b=False), z1, "silu", offsets, e)
        grads["w1"] = grouped_grad_weight(dz1, us, offsets, e)
        dus = grouped(dz1, w["w1"], offsets, trans_b=False)
        du = torch.empty_like(x)  # the gradient of sending rows out is joining them unweighted
        dgt.gemm_combine(t, top, h, dt, dus, h, slot, None, None, 0, du, h, stream=stream())
        dz0, db0 = act_grad(du, z0, "gelu")
        grads["b0"] = db0[0]
        grads["w0"] = linear(dz0, x, trans_a=True, trans_b=False, out=torch.float32)
        dx = linear(dz0, w["w0"], trans_b=False, residual=dy)  # the residual stream's own gradient is dy
        return dx, dweights, grads

    def update(self, grads, rate):
        for k, g in grads.items():
            self.master[k] -= rate * g
        self.cast()


def choose(logits, top):
    """The `top` likeliest experts of every token and their weights."""
    p, ids = torch.topk(torch.softmax(logits, dim=1), top, dim=1)
    return ids.to(torch.int32), p / p.sum(1, keepdim=True)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=512)
    args = ap.parse_args()
    gen = torch.Generator().manual_seed(1)
    h, hidden, experts, top = 256, 512, 8, 2
    layer = ExpertLayer(h, hidden, experts)
    x = torch.randn(args.tokens, h, generator=gen).cuda().to(layer.dtype)
    ids, weights = choose(torch.randn(args.tokens, experts, generator=gen).cuda(), top)
    target = torch.randn(args.tokens, h, generator=gen).cuda()
    for step in range(args.steps):
        y, kept = layer.forward(x, ids, weights)
        error = y.float() - target
        if step % 5 == 0 or step == args.steps - 1:
            print(f"step {step}: loss {float((error * error).mean()):.4f}")
        _, _, grads = layer.backward((2.0 / args.tokens * error).to(layer.dtype), kept)
        layer.update(grads, 0.03)


if __name__ == "__main__":
    main()
