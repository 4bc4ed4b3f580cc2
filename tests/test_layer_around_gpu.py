"""The operators around a layer, together and as programs use them: a norm, a gate, experts and the
loss forward and backward against 64 bits; the same served with 4-bit weights; captured graphs,
streams of their own, and buffers past 32-bit offsets."""
import math

import pytest
import torch

from gpu_helpers import need_gpu, say
from layer_helpers import DEV, DT, U32, close, half_step, out, randn
from test_layer_w4_gpu import weights as w4_weights

pytestmark = pytest.mark.gpu


def workspace(nbytes):
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)


def test_training_step_of_norm_gate_experts_and_loss():
    """examples/expert_model.py against autograd in 64 bits, with the choices that the gate made."""
    need_gpu()
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import expert_model
    T, h, hidden, experts, top, V = 200, 64, 96, 8, 2, 500
    for score, bias in (("softmax", False), ("sigmoid", True)):
        say(f"expert_model {score}")
        model = expert_model.ExpertModel(h, hidden, experts, V, top=top, score=score, seed=3)
        gen = torch.Generator().manual_seed(4)
        if bias:
            model.bias = (0.1 * torch.randn(experts, generator=gen)).to(DEV)
        x = torch.randn(T, h, generator=gen).to(DEV, torch.bfloat16)
        labels = torch.randint(0, V, (T,), generator=gen).to(DEV, torch.int32)
        labels[::9] = -1
        loss, kept = model.forward(x, labels)
        dx, grads = model.backward(kept)
        torch.cuda.synchronize()
        ids = kept["ids"]
        # The same in 64 bits, from the same 16-bit weights.
        w = {k: v.double().requires_grad_(True) for k, v in model.w.items()}
        x64 = x.double().requires_grad_(True)
        mean = x64.mean(1, keepdim=True)
        u = (x64 - mean) / torch.sqrt(((x64 - mean) ** 2).mean(1, keepdim=True) + expert_model.EPS) * w["gamma"] + w["beta"]
        logits = u @ w["gate"].T
        s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
        p = s.gather(1, ids.long())
        p = p / p.sum(1, keepdim=True)
        y = x64
        for j in range(top):
            e = ids[:, j].long()
            z = torch.bmm(w["w1"][e], u[:, :, None])[:, :, 0] + w["b1"][e]
            y = y + p[:, j:j + 1] * torch.bmm(w["w2"][e], (z * torch.sigmoid(z))[:, :, None])[:, :, 0]
        L = y @ w["out"].T
        has = labels >= 0
        each = torch.logsumexp(L, 1) - L.gather(1, labels.clamp(min=0).long()[:, None])[:, 0]
        want = (each * has).sum() / has.sum()
        got = torch.autograd.grad(want, [x64] + list(w.values()))
        # Every intermediate is rounded to bf16 once (half a step of 2^-8): about ten of them in a row, whose
        # errors are independent, stay below a twentieth of each gradient's norm.
        want = float(want.detach())
        assert abs(float(loss) - want) < 0.02 * abs(want)
        for name, a, b in [("x", dx, got[0])] + [(k, grads[k], g) for k, g in zip(w, got[1:])]:
            err = (a.double() - b).norm() / b.norm()
            assert err < 0.05, (score, name, float(err))


def test_experts_served_with_4_bit_weights():
    """A decoding batch: norm, gate, rows sent out, experts of 4-bit weights, rows joined."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(5)
    T, h, hidden, E, top, group = 12, 128, 256, 6, 2, 32
    s = torch.cuda.current_stream()
    x = randn(gen, T, h, dtype="bf16")
    c1, s1, _, v1, _ = w4_weights(gen, (E, hidden), h, group, False, "bf16")
    c2, s2, z2, v2, _ = w4_weights(gen, (E, h), hidden, group, True, "bf16")
    wg = randn(gen, E, h, dtype="bf16")
    u, logits = out(T, h, dtype="bf16"), out(T, E)
    dgt.gemm_norm(T, h, "bf16", x, h, None, None, 1e-5, u, h, stream=s)
    dgt.gemm_linear(T, E, h, "bf16", 0, 1, u, h, wg, h, None, "none", None, 0, logits, E, "f32", stream=s)
    ids, w = torch.empty(T, top, dtype=torch.int32, device=DEV), out(T, top)
    dgt.gemm_gate(T, E, top, "f32", logits, E, "softmax", None, 1, 1, 1, True, 1.0, ids, w, stream=s)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    order, slot = (torch.empty(T * top, dtype=torch.int32, device=DEV) for _ in range(2))
    size = dgt.gemm_route_workspace(T, top, E)
    dgt.gemm_route(T, top, E, ids, off, order, slot, workspace(size), size, stream=s)
    us, a, ys = out(T * top, h, dtype="bf16"), out(T * top, hidden, dtype="bf16"), out(T * top, h, dtype="bf16")
    dgt.gemm_dispatch(T, top, h, "bf16", u, h, slot, us, h, stream=s)
    dgt.gemm_grouped_w4(E, T * top, hidden, h, "bf16", off, us, h, c1, h, hidden * h, s1, None, h // group, hidden * h // group,
                        group, None, "silu", None, 0, a, hidden, "bf16", stream=s)
    dgt.gemm_grouped_w4(E, T * top, h, hidden, "bf16", off, a, hidden, c2, hidden, h * hidden, s2, z2, hidden // group,
                        h * hidden // group, group, None, "none", None, 0, ys, h, "bf16", stream=s)
    y = out(T, h, dtype="bf16")
    dgt.gemm_combine(T, top, h, "bf16", ys, h, slot, w, x, h, y, h, stream=s)
    torch.cuda.synchronize()
    u64, want = u.double(), x.double().clone()
    p = torch.softmax(logits.double(), 1)
    assert torch.equal(ids.long(), torch.topk(p, top, dim=1).indices)
    p = p.gather(1, ids.long())
    p = p / p.sum(1, keepdim=True)
    size = x.double().abs()
    for j in range(top):
        e = ids[:, j].long()
        z = torch.bmm(v1[e], u64[:, :, None])[:, :, 0]
        act = z * torch.sigmoid(z)
        want += p[:, j:j + 1] * torch.bmm(v2[e], act[:, :, None])[:, :, 0]
        size += p[:, j:j + 1] * torch.bmm(v2[e].abs(), act.abs()[:, :, None])[:, :, 0]
    # `a` and `ys` are rounded to bf16, and y; float32 sums are far below that.
    close(y, want, 3 * half_step("bf16") * size + 1e-5, "y")


CALLS = {}


def call(f):
    CALLS[f.__name__] = f
    return f


@call
def norm(dgt, gen):
    M, N = 300, 520
    x, dy, g = randn(gen, M, N, dtype="bf16"), randn(gen, M, N, dtype="bf16"), randn(gen, 1, N, dtype="bf16")[0]
    y, mean, rstd, dx, dg, db = (torch.empty_like(x), out(1, M)[0], out(1, M)[0], torch.empty_like(x), out(1, N)[0],
                                 out(1, N)[0])
    size = dgt.gemm_norm_grad_workspace(M, N)
    ws = workspace(size)

    def run(s):
        dgt.gemm_norm(M, N, "bf16", x, N, g, None, 1e-5, y, N, mean, rstd, stream=s)
        dgt.gemm_norm_grad(M, N, "bf16", dy, N, x, N, g, mean, rstd, None, 0, dx, N, dg, db, ws, size, stream=s)
    return run, [x, dy], [y, mean, rstd, dx, dg, db]


@call
def gate(dgt, gen):
    T, E, top = 500, 64, 6
    L, b, dw = randn(gen, T, E), 0.1 * randn(gen, 1, E)[0], randn(gen, T, top)
    ids, w, dl = torch.empty(T, top, dtype=torch.int32, device=DEV), out(T, top), out(T, E)

    def run(s):
        dgt.gemm_gate(T, E, top, "f32", L, E, "sigmoid", b, 8, 4, 2, True, 2.5, ids, w, stream=s)
        dgt.gemm_gate_grad(T, E, top, "f32", L, E, "sigmoid", True, 2.5, ids, dw, dl, E, stream=s)
    return run, [L, dw], [ids, w, dl]


@call
def w4(dgt, gen):
    M, N, K = 5, 96, 256
    x = randn(gen, M, K, dtype="f16")
    codes, s, z, _, _ = w4_weights(gen, (3, N), K, 64, True, "f16")
    y, yg = out(M, N, dtype="f16"), out(M, N, dtype="f16")
    off = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device=DEV)

    def run(stream):
        dgt.gemm_linear_w4(M, N, K, "f16", x, K, codes, K, s, z, 4, 64, None, "gelu", None, 0, y, N, "f16", stream=stream)
        dgt.gemm_grouped_w4(3, M, N, K, "f16", off, x, K, codes, K, N * K, s, z, 4, N * 4, 64, None, "none", None, 0, yg, N,
                            "f16", stream=stream)
    return run, [x], [y, yg]


def loss_call(T, V, H):
    def make(dgt, gen):
        x, w = randn(gen, T, H, dtype="bf16"), randn(gen, V, H, dtype="bf16", scale=H ** -0.5)
        labels = torch.randint(0, V, (T,), generator=gen).to(DEV, torch.int32)
        dloss = randn(gen, 1, T)[0]
        found, lse, dx, dw = out(1, T)[0], out(1, T)[0], out(T, H, dtype="bf16"), out(V, H)
        n1, n2 = dgt.gemm_loss_workspace(T, V, H), dgt.gemm_loss_grad_workspace(T, V, H)
        w1, w2 = workspace(n1), workspace(n2)

        def run(s):
            dgt.gemm_loss(T, V, H, "bf16", x, H, w, H, labels, found, lse, w1, n1, stream=s)
            dgt.gemm_loss_grad(T, V, H, "bf16", x, H, w, H, labels, lse, dloss, dx, H, dw, H, "f32", False, w2, n2, stream=s)
        return run, [x, w, dloss], [found, lse, dx, dw]
    return make


CALLS["loss_few"] = loss_call(20, 700, 64)
CALLS["loss_tiles"] = loss_call(301, 3000, 128)


@pytest.mark.parametrize("name", list(CALLS))
def test_captured_and_replayed(name):
    """Replays on other inputs, with eager work between them, against eager calls, bit for bit."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    say(f"graph of {name}")
    gen = torch.Generator().manual_seed(6)
    run, inputs, outputs = CALLS[name](dgt, gen)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(side)  # loads the kernels
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(torch.cuda.current_stream())
    for turn in range(4):
        for x in inputs:
            x.copy_((torch.randn(x.shape, generator=gen) * (0.1 if x.dim() == 2 and x.shape[0] > 600 else 1)).to(x.dtype))
        for o in outputs:
            o.fill_(-3 if o.dtype == torch.int32 else float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outputs]
        for o in outputs:
            o.fill_(-3 if o.dtype == torch.int32 else float("nan"))
        run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        for a, b in zip(got, outputs):
            assert torch.equal(a, b), (name, turn)


@pytest.mark.parametrize("name", list(CALLS))
def test_streams_of_their_own(name):
    """Two streams at once, each with buffers and a workspace of its own, ordered by the stream alone."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    gen = torch.Generator().manual_seed(7)
    calls = [CALLS[name](dgt, gen) for _ in range(2)]
    want = []
    for run, _, outputs in calls:
        run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([o.clone() for o in outputs])
        for o in outputs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for (run, _, _), s in zip(calls, streams):
            run(s)
    for s in streams:
        s.synchronize()
    for (_, _, outputs), w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outputs, w)), name


def test_past_32_bit_offsets():
    """Rows, logits and codes whose offsets pass 2^31 bytes and 2^31 elements: the last rows against the
    same rows by themselves."""
    need_gpu()
    import dense_gemm_tile_amd as dgt
    s = torch.cuda.current_stream()
    gen = torch.Generator().manual_seed(8)
    say("norm past 2^31 elements")
    M, N, pitch = 5, 300, 1 << 29
    x = torch.zeros(4 * pitch + N, dtype=torch.bfloat16, device=DEV)
    rows = torch.as_strided(x, (M, N), (pitch, 1))
    rows.copy_(torch.randn(M, N, generator=gen))
    y, one = out(M, N, dtype="bf16"), out(M, N, dtype="bf16")
    mean, rstd = out(1, M)[0], out(1, M)[0]
    dgt.gemm_norm(M, N, "bf16", x, pitch, None, None, 1e-5, y, N, mean, rstd, stream=s)
    small = rows.contiguous()
    dgt.gemm_norm(M, N, "bf16", small, N, None, None, 1e-5, one, N, stream=s)
    assert torch.equal(y, one)
    dy = randn(gen, M, N, dtype="bf16")
    d1, d2 = out(M, N, dtype="bf16"), out(M, N, dtype="bf16")
    size = dgt.gemm_norm_grad_workspace(M, N)
    for src, ld, to in ((x, pitch, d1), (small, N, d2)):
        dgt.gemm_norm_grad(M, N, "bf16", dy, N, src, ld, None, mean, rstd, None, 0, to, N, None, None, None, 0, stream=s)
    assert torch.equal(d1, d2)
    say("gate past 2^31 elements")
    L = torch.as_strided(x, (M, 64), (pitch, 1))
    ids, w = torch.empty(M, 4, dtype=torch.int32, device=DEV), out(M, 4)
    ids2, w2 = torch.empty_like(ids), out(M, 4)
    dgt.gemm_gate(M, 64, 4, "bf16", x, pitch, "softmax", None, 1, 1, 1, False, 1.0, ids, w, stream=s)
    dgt.gemm_gate(M, 64, 4, "bf16", L.contiguous(), 64, "softmax", None, 1, 1, 1, False, 1.0, ids2, w2, stream=s)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    del x, rows, L
    say("w4 past 2^31 bytes")
    N, K = 70000, 65536
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    sc = torch.rand(N, K // 128, device=DEV).to(torch.bfloat16)
    a = randn(gen, 3, K, dtype="bf16")
    y = out(3, N, dtype="f32")
    dgt.gemm_linear_w4(3, N, K, "bf16", a, K, codes, K, sc, None, K // 128, 128, None, "none", None, 0, y, N, "f32", stream=s)
    last = out(3, 48, dtype="f32")
    c2, s2 = codes[-48:].clone(), sc[-48:].clone()
    dgt.gemm_linear_w4(3, 48, K, "bf16", a, K, c2, K, s2, None, K // 128, 128, None, "none", None, 0, last, 48, "f32", stream=s)
    want = out(3, 48)
    q = torch.stack([c2 & 15, c2 >> 4], -1).reshape(48, K).double() - 8
    wv = q * s2.double().repeat_interleave(128, 1)
    tol = (128 + K // 128 + 16) * U32 * (a.double().abs() @ (s2.double().repeat_interleave(128, 1) * (40 + q.abs() + 8)).T)
    close(y[:, -48:], a.double() @ wv.T, tol, "Y")
    close(last, a.double() @ wv.T, tol, "the last columns")
