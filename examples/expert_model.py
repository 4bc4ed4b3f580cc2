"""A small model of experts trained through the layer operators: tokens pass a norm, a gate sends each to
`top` of E experts (two products with SiLU between them), their outputs are joined onto the residual
stream, and an output layer's cross entropy closes it. Forward pass, gradients and plain gradient
descent, on one GPU.

    python examples/expert_model.py [--steps 40] [--tokens 512] [--score softmax|sigmoid]

prints the loss of every fifth step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_tile_amd as dgt  # noqa: E402
from expert_layer import DTYPE, act_grad, grouped, grouped_grad_weight, linear, stream  # noqa: E402

EPS = 1e-5


def workspace(size, like):
    return torch.empty(max(size, 1), dtype=torch.uint8, device=like.device)


class ExpertModel:
    """Weights in 16 bits, float32 masters beside them for the update."""

    def __init__(self, h, hidden, experts, vocabulary, top=2, score="softmax", dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.top, self.score, self.dtype = top, score, dtype
        self.bias = None  # of the choice: float32, one for each expert
        draw = lambda *s: (torch.randn(*s, generator=gen) * s[-1] ** -0.5).to(device)  # noqa: E731
        self.master = {"gamma": torch.ones(h, device=device), "beta": torch.zeros(h, device=device), "gate": draw(experts, h),
                       "w1": draw(experts, hidden, h), "b1": torch.zeros(experts, hidden, device=device),
                       "w2": draw(experts, h, hidden), "out": draw(vocabulary, h)}
        self.cast()

    def cast(self):
        self.w = {k: v.to(self.dtype) for k, v in self.master.items()}

    def forward(self, x, labels):
        """x: T x h; labels: T int32, -1 for none. Returns the mean loss and what the backward pass
        needs."""
        w, (t, h), dt, top, e = self.w, x.shape, DTYPE[x.dtype], self.top, self.w["gate"].shape[0]
        new = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=x.device)  # noqa: E731
        u, mean, rstd = torch.empty_like(x), new(t), new(t)
        dgt.gemm_norm(t, h, dt, x, h, w["gamma"], w["beta"], EPS, u, h, mean, rstd, stream=stream())
        logits = linear(u, w["gate"], out=torch.float32)
        ids, weights = new(t, top, dtype=torch.int32), new(t, top)
        dgt.gemm_gate(t, e, top, "f32", logits, e, self.score, self.bias, 1, 1, 1, True, 1.0, ids, weights, stream=stream())
        offsets, order, slot = (new(n, dtype=torch.int32) for n in (e + 1, t * top, t * top))
        size = dgt.gemm_route_workspace(t, top, e)
        dgt.gemm_route(t, top, e, ids, offsets, order, slot, workspace(size, x), size, stream=stream())
        us, y = new(t * top, h, dtype=x.dtype), torch.empty_like(x)
        dgt.gemm_dispatch(t, top, h, dt, u, h, slot, us, h, stream=stream())
        a, z = grouped(us, w["w1"], offsets, w["b1"], act="silu", keep_z=True)
        ys = grouped(a, w["w2"], offsets)
        dgt.gemm_combine(t, top, h, dt, ys, h, slot, weights, x, h, y, h, stream=stream())
        v = w["out"].shape[0]
        loss, lse = new(t), new(t)
        size = dgt.gemm_loss_workspace(t, v, h)
        dgt.gemm_loss(t, v, h, dt, y, h, w["out"], h, labels, loss, lse, workspace(size, x), size, stream=stream())
        count = (labels >= 0).sum().clamp(min=1)
        return loss.sum() / count, dict(x=x, u=u, mean=mean, rstd=rstd, logits=logits, ids=ids, weights=weights, offsets=offsets,
                                        slot=slot, us=us, a=a, z=z, ys=ys, y=y, labels=labels, lse=lse, count=count)

    def backward(self, k):
        """Gradients of x and of every parameter, of the mean loss."""
        w, x, (t, h), dt = self.w, k["x"], k["x"].shape, DTYPE[k["x"].dtype]
        top, e, v = self.top, w["gate"].shape[0], w["out"].shape[0]
        new = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=x.device)  # noqa: E731
        grads, dy = {"out": new(v, h)}, torch.empty_like(x)
        dloss = (1.0 / k["count"]).to(torch.float32).expand(t).contiguous()
        size = dgt.gemm_loss_grad_workspace(t, v, h)
        dgt.gemm_loss_grad(t, v, h, dt, k["y"], h, w["out"], h, k["labels"], k["lse"], dloss, dy, h, grads["out"], h, "f32", False,
                           workspace(size, x), size, stream=stream())
        dys, dweights = torch.empty_like(k["ys"]), torch.empty_like(k["weights"])
        dgt.gemm_combine_grad(t, top, h, dt, dy, h, k["ys"], h, k["slot"], k["weights"], dys, h, dweights, stream=stream())
        grads["w2"] = grouped_grad_weight(dys, k["a"], k["offsets"], e)
        dz, grads["b1"] = act_grad(grouped(dys, w["w2"], k["offsets"], trans_b=False), k["z"], "silu", k["offsets"], e)
        grads["w1"] = grouped_grad_weight(dz, k["us"], k["offsets"], e)
        dus, du = grouped(dz, w["w1"], k["offsets"], trans_b=False), torch.empty_like(x)
        dgt.gemm_combine(t, top, h, dt, dus, h, k["slot"], None, None, 0, du, h, stream=stream())
        dlogits = new(t, e)
        dgt.gemm_gate_grad(t, e, top, "f32", k["logits"], e, self.score, True, 1.0, k["ids"], dweights, dlogits, e, stream=stream())
        dlogits = dlogits.to(x.dtype)
        grads["gate"] = linear(dlogits, k["u"], trans_a=True, trans_b=False, out=torch.float32)
        du = linear(dlogits, w["gate"], trans_b=False, residual=du)
        dx, grads["gamma"], grads["beta"] = torch.empty_like(x), new(h), new(h)
        size = dgt.gemm_norm_grad_workspace(t, h)
        dgt.gemm_norm_grad(t, h, dt, du, h, x, h, w["gamma"], k["mean"], k["rstd"], dy, h, dx, h, grads["gamma"], grads["beta"],
                           workspace(size, x), size, stream=stream())  # (dy: what went past the norm)
        return dx, grads

    def update(self, grads, rate):
        for k, g in grads.items():
            self.master[k] -= rate * g
        self.cast()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--score", choices=["softmax", "sigmoid"], default="softmax")
    args = ap.parse_args()
    gen = torch.Generator().manual_seed(1)
    h, hidden, experts, vocabulary = 256, 512, 8, 1000
    model = ExpertModel(h, hidden, experts, vocabulary, score=args.score)
    x = torch.randn(args.tokens, h, generator=gen).cuda().to(model.dtype)
    labels = torch.randint(0, vocabulary, (args.tokens,), generator=gen).to(torch.int32).cuda()
    for step in range(args.steps):
        loss, kept = model.forward(x, labels)
        if step % 5 == 0 or step == args.steps - 1:
            print(f"step {step}: loss {float(loss):.4f}")
        _, grads = model.backward(kept)
        model.update(grads, 2.0)


if __name__ == "__main__":
    main()
