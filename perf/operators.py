"""The layer operators that are timed: fused linear layers, tokens sent to experts and
back, and the experts' products. Each has its plain form in elementary torch operations
(`own` false) and the library's calls (`own` true), on the same prepared state.

Operators and what they return:

  linear            Y = act(X @ W' + bias) + R; also Z = X @ W' + bias when it is kept for
                    the backward pass
  linear_backward   of the same layer, from dY and Z: dX, dW and dbias
  dispatch          expert ids -> offsets, order and slots of the tokens sorted by expert,
                    and the gathered rows; with `grad`, also the rows' gradient sent back
  combine           rows weighted and summed per token, plus R; with `grad`, also the
                    gradients of the rows and of the weights
  experts           the linear layer with one weight matrix per group of sorted rows
  experts_backward  of the same layer: dX, dW and dbias of every expert
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"


def listed():
    return [
        # One token through an output projection: the weights are read once, latency counts.
        dict(name="linear_token", op="linear", m=1, n=4096, k=4096, dtype="bf16", out="bf16", layout="nt",
             act="none", bias=False, residual=True, keep_z=False, pad=0),
        # A batch of decoding sequences through a wide up-projection.
        dict(name="linear_decode", op="linear", m=48, n=8192, k=8192, dtype="f16", out="f16", layout="nt",
             act="gelu", bias=True, residual=False, keep_z=False, pad=0),
        # A prompt whose length and widths fill no tile.
        dict(name="linear_ragged", op="linear", m=4097, n=1000, k=1032, dtype="f16", out="f16", layout="nt",
             act="gelu", bias=True, residual=True, keep_z=False, pad=0),
        # A training forward at the widest size: Z is kept for the backward pass.
        dict(name="linear_train", op="linear", m=8192, n=8192, k=8192, dtype="bf16", out="bf16", layout="nt",
             act="silu", bias=True, residual=False, keep_z=True, pad=0),
        # Its backward pass at an ordinary size.
        dict(name="linear_backward", op="linear_backward", m=4096, n=4096, k=4096, dtype="bf16", layout="nt",
             act="gelu", pad=0),
        # A decoding batch sent to its experts: nothing but latency.
        dict(name="dispatch_decode", op="dispatch", t=32, top=4, e=64, h=2048, dtype="bf16", grad=False, drop=0.0),
        # A training batch sent to its experts, some choices dropped, with the gradient.
        dict(name="dispatch_train", op="dispatch", t=16384, top=4, e=64, h=4096, dtype="bf16", grad=True, drop=0.05),
        # A decoding batch's expert outputs joined onto the residual stream.
        dict(name="combine_decode", op="combine", t=32, top=4, e=64, h=2048, dtype="bf16", residual=True, grad=False,
             drop=0.0),
        # The same in training, with the gradients of rows and weights.
        dict(name="combine_train", op="combine", t=16384, top=4, e=64, h=4096, dtype="f16", residual=True, grad=True,
             drop=0.05),
        # A decoding batch's choices: a few rows for each of many experts.
        dict(name="experts_decode", op="experts", t=32, top=4, e=64, n=2048, k=2048, dtype="bf16", out="bf16",
             layout="nt", act="silu", bias=False, keep_z=False),
        # A long prompt or training batch: about a thousand rows an expert, unevenly.
        dict(name="experts_train", op="experts", t=16384, top=2, e=32, n=4096, k=2048, dtype="bf16", out="bf16",
             layout="nt", act="gelu", bias=True, keep_z=True),
        # The backward pass of experts of uneven load.
        dict(name="experts_backward", op="experts_backward", t=8192, top=2, e=16, n=2048, k=2048, dtype="f16",
             layout="nt", act="silu"),
    ]


def _spread(rng, lo, hi, step=1):
    """A size of [lo, hi], spread over its logarithm, on a multiple of step where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v - v % step if v >= step else v))


def _width(rng, lo, hi):
    """A row width: mostly whole 16-byte pieces, now and then any number."""
    return _spread(rng, lo, hi, rng.choice([8, 8, 64, 128, 1]))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "dispatch", "combine", "experts", "experts",
                     "experts_backward"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]))
    act = rng.choice(["none", "relu", "gelu", "gelu_erf", "silu"])
    layout = rng.choice(["nt", "nt", "nn"])
    if op == "linear":
        case.update(m=_spread(rng, 1, 8192), n=_width(rng, 64, 8192), k=_width(rng, 64, 8192),
                    out=rng.choice([case["dtype"], case["dtype"], "f32"]), layout=layout, act=act,
                    bias=rng.random() < 0.6, residual=rng.random() < 0.5, keep_z=rng.random() < 0.3,
                    pad=rng.choice([0, 0, 8, 64, 3]))
    elif op == "linear_backward":
        case.update(m=_spread(rng, 1, 8192), n=_width(rng, 64, 4096), k=_width(rng, 64, 4096), layout=layout, act=act,
                    pad=rng.choice([0, 0, 8]))
    elif op in ("dispatch", "combine"):
        top = rng.choice([1, 2, 4, 8])
        h = _width(rng, 64, 4096)
        case.update(t=_spread(rng, 1, min(16384, 16384 * 4096 * 4 // (top * h))), top=top,
                    e=max(top, _spread(rng, 2, 256)), h=h, grad=rng.random() < 0.5, drop=rng.choice([0.0, 0.0, 0.1]))
        if op == "combine":
            case.update(residual=rng.random() < 0.5)
    else:
        top = rng.choice([1, 2, 4, 8])
        n, k = _width(rng, 64, 4096), _width(rng, 64, 2048)
        e = max(top, min(_spread(rng, 2, 128), 64 * 4096 * 2048 // (n * k)))
        t = _spread(rng, 1, (32768 if op == "experts" else 16384) // top)
        case.update(t=t, top=top, e=e, n=n, k=k, layout=layout, act=act)
        if op == "experts":
            case.update(out=rng.choice([case["dtype"], case["dtype"], "f32"]), bias=rng.random() < 0.6,
                        keep_z=rng.random() < 0.3)
    return case


def _randn(gen, shape, dtype, scale=1.0, pad=0):
    """Normal values in the first shape[-1] columns of rows that are `pad` elements wider."""
    shape = list(shape)
    wide = shape[:-1] + [shape[-1] + pad]
    x = torch.randn(wide, generator=gen, device=DEVICE, dtype=torch.float32).mul_(scale).to(dtype)
    return x[..., :shape[-1]]


def _choices(gen, t, top, e, drop):
    """`top` different experts a token, some experts liked more, and a share of choices dropped (-1)."""
    liked = 0.3 * torch.randn(e, generator=gen, device=DEVICE)
    noise = torch.rand(t, e, generator=gen, device=DEVICE).clamp_(1e-9, 1 - 1e-7)
    ids = torch.topk(liked - torch.log(-torch.log(noise)), top, dim=1).indices.to(torch.int32)
    if drop:
        ids[torch.rand(t, top, generator=gen, device=DEVICE) < drop] = -1
    return ids.contiguous()


def _sorted_by_expert(ids, e):
    """Offsets, order and slots of the choices sorted by expert, those dropped last (slot -1)."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, e), flat)
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(e, device=key.device)).sum(0)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=key.device)
    offsets[1:] = counts.cumsum(0)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=key.device)
    slot = torch.where(flat < 0, torch.full_like(slot, -1), slot)
    return offsets.to(torch.int32), order.to(torch.int32), slot.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, s = case["op"], dict(case)
    if op in ("linear", "linear_backward"):
        m, n, k, pad = case["m"], case["n"], case["k"], case["pad"]
        s["x"] = _randn(gen, (m, k), dt, pad=pad)
        s["w"] = _randn(gen, (n, k) if case["layout"] == "nt" else (k, n), dt, 1.0 / math.sqrt(k))
        if op == "linear":
            out = DTYPES[case["out"]]
            s["b"] = _randn(gen, (n,), dt, 0.5) if case["bias"] else None
            s["r"] = _randn(gen, (m, n), out) if case["residual"] else None
            s["y"] = torch.empty(m, n, dtype=out, device=DEVICE)
            s["z"] = torch.empty(m, n, dtype=dt, device=DEVICE) if case["keep_z"] else None
        else:
            s["z"] = _randn(gen, (m, n), dt)
            s["dy"] = _randn(gen, (m, n), dt, pad=pad)
            s["dz"] = torch.empty(m, n, dtype=dt, device=DEVICE)
            s["dx"] = torch.empty(m, k, dtype=dt, device=DEVICE)
            s["dw"] = torch.empty_like(s["w"])
            s["db"] = torch.empty(n, dtype=torch.float32, device=DEVICE)
        return s
    t, top, e = case["t"], case["top"], case["e"]
    ids = _choices(gen, t, top, e, case.get("drop", 0.0))
    rows = t * top
    if op == "dispatch":
        s["ids"] = ids
        s["x"] = _randn(gen, (t, case["h"]), dt)
        s["offsets"] = torch.empty(e + 1, dtype=torch.int32, device=DEVICE)
        s["order"] = torch.empty(rows, dtype=torch.int32, device=DEVICE)
        s["slot"] = torch.empty(t, top, dtype=torch.int32, device=DEVICE)
        s["xs"] = torch.zeros(rows, case["h"], dtype=dt, device=DEVICE)
        if case["grad"]:
            s["dxs"] = _randn(gen, (rows, case["h"]), dt)
            s["dx"] = torch.empty(t, case["h"], dtype=dt, device=DEVICE)
        return s
    offsets, _, slot = _sorted_by_expert(ids, e)
    if op == "combine":
        h = case["h"]
        s["slot"] = slot.reshape(t, top)
        s["weights"] = torch.softmax(torch.randn(t, top, generator=gen, device=DEVICE), dim=1)
        s["ys"] = _randn(gen, (rows, h), dt)
        s["r"] = _randn(gen, (t, h), dt) if case["residual"] else None
        s["y"] = torch.empty(t, h, dtype=dt, device=DEVICE)
        if case["grad"]:
            s["dy"] = _randn(gen, (t, h), dt)
            s["dys"] = torch.zeros(rows, h, dtype=dt, device=DEVICE)
            s["dw"] = torch.empty(t, top, dtype=torch.float32, device=DEVICE)
        return s
    n, k = case["n"], case["k"]
    s["offsets"], s["rows"] = offsets, rows
    s["capacity"] = int((offsets[1:] - offsets[:-1]).max())  # the most rows that an expert has
    s["x"] = _randn(gen, (rows, k), dt)
    s["w"] = _randn(gen, (e, n, k) if case["layout"] == "nt" else (e, k, n), dt, 1.0 / math.sqrt(k))
    if op == "experts":
        out = DTYPES[case["out"]]
        s["b"] = _randn(gen, (e, n), dt, 0.5) if case["bias"] else None
        s["y"] = torch.empty(rows, n, dtype=out, device=DEVICE)
        s["z"] = torch.empty(rows, n, dtype=dt, device=DEVICE) if case["keep_z"] else None
    else:
        s["z"] = _randn(gen, (rows, n), dt)
        s["dy"] = _randn(gen, (rows, n), dt)
        s["dz"] = torch.empty(rows, n, dtype=dt, device=DEVICE)
        s["dx"] = torch.empty(rows, k, dtype=dt, device=DEVICE)
        s["dw"] = torch.empty_like(s["w"])
        s["db"] = torch.empty(e, n, dtype=torch.float32, device=DEVICE)
    return s


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ plain forms

SQRT_2_OVER_PI = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(SQRT_2_OVER_PI * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        th = torch.tanh(SQRT_2_OVER_PI * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * SQRT_2_OVER_PI * (1 + 3 * 0.044715 * z * z)
    if act == "gelu_erf":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return torch.ones_like(z)


def _plain_linear(s):
    w = s["w"].float()
    z = s["x"].float() @ (w.t() if s["layout"] == "nt" else w)
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(DTYPES[s["out"]])
    return (y, z.to(s["x"].dtype)) if s["keep_z"] else (y,)


def _plain_linear_backward(s):
    dt = s["x"].dtype
    g = s["dy"].float() * _act_slope(s["z"].float(), s["act"])
    w, x = s["w"].float(), s["x"].float()
    nt = s["layout"] == "nt"
    dx = (g @ (w if nt else w.t())).to(dt)
    dw = (g.t() @ x if nt else x.t() @ g).to(dt)
    return dx, dw, g.sum(0)


def _sum_rows(rows, slot, weights=None):
    """Sum over each token's choices of their rows, in 32 bits, dropped ones left out."""
    kept = (slot >= 0).float()
    if weights is not None:
        kept = kept * weights
    return (rows[slot.clamp(min=0).long()].float() * kept[:, :, None]).sum(1)


def _plain_dispatch(s):
    offsets, order, slot = _sorted_by_expert(s["ids"], s["e"])
    rows = order.numel()
    kept = torch.arange(rows, device=order.device) < offsets[-1]
    xs = s["x"][(order // s["top"]).long()] * kept[:, None]
    slot = slot.reshape(s["t"], s["top"])
    if not s["grad"]:
        return offsets, order, slot, xs
    return offsets, order, slot, xs, _sum_rows(s["dxs"], slot).to(s["x"].dtype)


def _plain_combine(s):
    slot, ys = s["slot"], s["ys"]
    y = _sum_rows(ys, slot, s["weights"])
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(ys.dtype)
    if not s["grad"]:
        return (y,)
    at, kept = slot.clamp(min=0).long(), slot >= 0
    dy = s["dy"].float()
    dw = (ys[at].float() * dy[:, None, :]).sum(-1) * kept
    spare = torch.where(kept, at, torch.full_like(at, ys.shape[0]))  # dropped choices go to a spare row
    dys = torch.zeros(ys.shape[0] + 1, ys.shape[1], dtype=ys.dtype, device=ys.device)
    dys[spare.reshape(-1)] = (dy[:, None, :] * s["weights"][:, :, None]).to(ys.dtype).reshape(-1, ys.shape[1])
    return y, dys[:-1], dw


def _padded_place(s):
    """Of each sorted row: its expert, and its place where every expert has `capacity` rows."""
    at = torch.arange(s["rows"], device=s["x"].device)
    expert = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return expert, expert * s["capacity"] + at - s["offsets"].long()[expert]


def _padded(s, x, place):
    wide = torch.zeros(s["e"] * s["capacity"], x.shape[1], dtype=torch.float32, device=x.device)
    wide[place] = x
    return wide.view(s["e"], s["capacity"], x.shape[1])


def _plain_experts(s):
    expert, place = _padded_place(s)
    w = s["w"].float()
    z = torch.bmm(_padded(s, s["x"].float(), place), w.transpose(1, 2) if s["layout"] == "nt" else w)
    z = z.view(-1, s["n"])[place]
    if s["b"] is not None:
        z = z + s["b"].float()[expert]
    y = _act(z, s["act"]).to(DTYPES[s["out"]])
    return (y, z.to(s["x"].dtype)) if s["keep_z"] else (y,)


def _plain_experts_backward(s):
    dt = s["x"].dtype
    _, place = _padded_place(s)
    g = _padded(s, s["dy"].float() * _act_slope(s["z"].float(), s["act"]), place)
    x, w = _padded(s, s["x"].float(), place), s["w"].float()
    nt = s["layout"] == "nt"
    dx = torch.bmm(g, w if nt else w.transpose(1, 2)).view(-1, s["k"])[place].to(dt)
    dw = (torch.bmm(g.transpose(1, 2), x) if nt else torch.bmm(x.transpose(1, 2), g)).to(dt)
    return dx, dw, g.sum(1)


PLAIN = {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "dispatch": _plain_dispatch,
         "combine": _plain_combine, "experts": _plain_experts, "experts_backward": _plain_experts_backward}


# ---------------------------------------------------------- the library's calls

def _ld(x):
    return 0 if x is None else x.stride(-2)


def _own_linear(s):
    import dense_gemm_tile_amd as dgt
    x, w, r, y, z = s["x"], s["w"], s["r"], s["y"], s["z"]
    dgt.gemm_linear(s["m"], s["n"], s["k"], s["dtype"], 0, s["layout"] == "nt", x, _ld(x), w, _ld(w), s["b"], s["act"],
                    r, _ld(r), y, _ld(y), s["out"], z, _ld(z), stream=torch.cuda.current_stream())
    return (y, z) if s["keep_z"] else (y,)


def _own_linear_backward(s):
    import dense_gemm_tile_amd as dgt
    m, n, k, dt = s["m"], s["n"], s["k"], s["dtype"]
    x, w, z, dy, dz, dx, dw, db = (s[q] for q in ("x", "w", "z", "dy", "dz", "dx", "dw", "db"))
    stream = torch.cuda.current_stream()
    size = dgt.gemm_act_grad_workspace(1, m, n)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    dgt.gemm_act_grad(1, m, n, dt, s["act"], None, dy, _ld(dy), z, _ld(z), dz, _ld(dz), db, ws, size, stream=stream)
    nt = s["layout"] == "nt"
    dgt.gemm_linear(m, k, n, dt, 0, not nt, dz, _ld(dz), w, _ld(w), None, "none", None, 0, dx, _ld(dx), dt,
                    stream=stream)
    if nt:
        dgt.gemm_linear(n, k, m, dt, 1, 0, dz, _ld(dz), x, _ld(x), None, "none", None, 0, dw, _ld(dw), dt,
                        stream=stream)
    else:
        dgt.gemm_linear(k, n, m, dt, 1, 0, x, _ld(x), dz, _ld(dz), None, "none", None, 0, dw, _ld(dw), dt,
                        stream=stream)
    return dx, dw, db


def _own_dispatch(s):
    import dense_gemm_tile_amd as dgt
    t, top, e, h, dt = s["t"], s["top"], s["e"], s["h"], s["dtype"]
    x, slot, xs = s["x"], s["slot"], s["xs"]
    stream = torch.cuda.current_stream()
    size = dgt.gemm_route_workspace(t, top, e)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    dgt.gemm_route(t, top, e, s["ids"], s["offsets"], s["order"], slot, ws, size, stream=stream)
    dgt.gemm_dispatch(t, top, h, dt, x, _ld(x), slot, xs, _ld(xs), stream=stream)
    if not s["grad"]:
        return s["offsets"], s["order"], slot, xs
    dxs, dx = s["dxs"], s["dx"]
    dgt.gemm_combine(t, top, h, dt, dxs, _ld(dxs), slot, None, None, 0, dx, _ld(dx), stream=stream)
    return s["offsets"], s["order"], slot, xs, dx


def _own_combine(s):
    import dense_gemm_tile_amd as dgt
    t, top, h, dt = s["t"], s["top"], s["h"], s["dtype"]
    ys, slot, w, r, y = s["ys"], s["slot"], s["weights"], s["r"], s["y"]
    stream = torch.cuda.current_stream()
    dgt.gemm_combine(t, top, h, dt, ys, _ld(ys), slot, w, r, _ld(r), y, _ld(y), stream=stream)
    if not s["grad"]:
        return (y,)
    dy, dys = s["dy"], s["dys"]
    dgt.gemm_combine_grad(t, top, h, dt, dy, _ld(dy), ys, _ld(ys), slot, w, dys, _ld(dys), s["dw"], stream=stream)
    return y, dys, s["dw"]


def _own_experts(s):
    import dense_gemm_tile_amd as dgt
    x, w, y, z = s["x"], s["w"], s["y"], s["z"]
    dgt.gemm_grouped(s["e"], s["rows"], s["n"], s["k"], s["dtype"], s["layout"] == "nt", s["offsets"], x, _ld(x), w,
                     _ld(w), w.stride(0), s["b"], s["act"], None, 0, y, _ld(y), s["out"], z, _ld(z),
                     stream=torch.cuda.current_stream())
    return (y, z) if s["keep_z"] else (y,)


def _own_experts_backward(s):
    import dense_gemm_tile_amd as dgt
    e, rows, n, k, dt = s["e"], s["rows"], s["n"], s["k"], s["dtype"]
    off, x, w, z, dy, dz, dx, dw, db = (s[q] for q in ("offsets", "x", "w", "z", "dy", "dz", "dx", "dw", "db"))
    stream = torch.cuda.current_stream()
    size = dgt.gemm_act_grad_workspace(e, rows, n)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    dgt.gemm_act_grad(e, rows, n, dt, s["act"], off, dy, _ld(dy), z, _ld(z), dz, _ld(dz), db, ws, size, stream=stream)
    nt = s["layout"] == "nt"
    dgt.gemm_grouped(e, rows, k, n, dt, not nt, off, dz, _ld(dz), w, _ld(w), w.stride(0), None, "none", None, 0, dx,
                     _ld(dx), dt, stream=stream)
    a, b = (dz, x) if nt else (x, dz)
    dgt.gemm_grouped_grad_weight(e, rows, a.shape[1], b.shape[1], dt, off, a, _ld(a), b, _ld(b), dw, _ld(dw),
                                 dw.stride(0), dt, False, stream=stream)
    return dx, dw, db


OWN = {"linear": _own_linear, "linear_backward": _own_linear_backward, "dispatch": _own_dispatch,
       "combine": _own_combine, "experts": _own_experts, "experts_backward": _own_experts_backward}


# ------------------------------------------------------------ work and definition

def work(case):
    """Bytes (each input read once, each output written once) and operations of one pass."""
    size = {"f16": 2, "bf16": 2, "f32": 4}
    d, op = size[case["dtype"]], case["op"]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        o = size[case["out"]]
        return {"bytes": d * (m * k + n * k + n * case["bias"] + m * n * case["keep_z"]) + o * m * n * (1 + case["residual"]),
                "flops": 2 * m * n * k}
    if op == "linear_backward":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": d * (2 * m * n + 2 * m * k + 2 * n * k) + 4 * n, "flops": 4 * m * n * k}
    t, top, e = case["t"], case["top"], case["e"]
    rows = t * top * (1 - case.get("drop", 0.0))
    if op == "dispatch":
        h = case["h"]
        both = 2 if case["grad"] else 1
        return {"bytes": int(d * h * (t + rows) * both + 4 * (3 * t * top + e + 1)), "flops": int((both - 1) * rows * h)}
    if op == "combine":
        h = case["h"]
        fwd = d * h * (rows + t * (1 + case["residual"])) + 8 * t * top
        bwd = (d * h * (rows + t) + 4 * t * top) if case["grad"] else 0
        return {"bytes": int(fwd + bwd), "flops": int(2 * rows * h * (2.5 if case["grad"] else 1))}
    n, k = case["n"], case["k"]
    used = e * (1 - (1 - 1 / e) ** rows)  # experts that get a row, were all liked alike
    if op == "experts":
        return {"bytes": int(d * (rows * k + used * n * k + used * n * case["bias"] + rows * n * case["keep_z"])
                             + size[case["out"]] * rows * n), "flops": int(2 * rows * n * k)}
    return {"bytes": int(d * (2 * rows * n + 2 * rows * k + (used + e) * n * k) + 4 * e * n), "flops": int(4 * rows * n * k)}


def _value64(z, act):
    """The activation and its slope, from their definitions, in 64 bits."""
    one = torch.ones_like(z)
    if act == "relu":
        return torch.maximum(z, 0 * z), torch.where(z > 0, one, 0 * z)
    if act == "gelu":  # z * sigmoid(v), v = 2 sqrt(2/pi) (z + 0.044715 z^3)
        v = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
        g = torch.sigmoid(v)
        return z * g, g + z * g * (1 - g) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z ** 2)
    if act == "gelu_erf":  # z times the normal distribution's function, whose slope is its density
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        g = torch.sigmoid(z)
        return z * g, g + z * g * (1 - g)
    return z, one


def exact(case, seed):
    s = prepare(case, seed)
    op, nt = case["op"], case.get("layout") == "nt"
    if op in ("linear", "linear_backward"):
        x, w = s["x"].double(), s["w"].double()
        wt = w.T if nt else w  # k x n
        if op == "linear":
            z = x @ wt + (0 if s["b"] is None else s["b"].double())
            y = _value64(z, case["act"])[0] + (0 if s["r"] is None else s["r"].double())
            return (y, z) if case["keep_z"] else (y,)
        g = s["dy"].double() * _value64(s["z"].double(), case["act"])[1]
        dwt = x.T @ g
        return g @ wt.T, dwt.T if nt else dwt, g.sum(0)
    if op == "dispatch":
        t, top, e = case["t"], case["top"], case["e"]
        flat = s["ids"].reshape(-1).tolist()
        lists = [[] for _ in range(e + 1)]
        for i, expert in enumerate(flat):
            lists[expert].append(i)  # -1: the last list
        offsets, order = [0], []
        for expert in range(e):
            order += lists[expert]
            offsets.append(len(order))
        kept = len(order)
        slot = [-1] * len(flat)
        for p, i in enumerate(order):
            slot[i] = p
        order += lists[e]
        whole = lambda v: torch.tensor(v, dtype=torch.int32, device=DEVICE)  # noqa: E731
        xs = torch.zeros_like(s["xs"], dtype=torch.float64)
        took = whole(order[:kept]).long()
        xs[:kept] = s["x"].double()[took // top]
        found = [whole(offsets), whole(order), whole(slot).reshape(t, top), xs]
        if case["grad"]:
            dx = torch.zeros(t, case["h"], dtype=torch.float64, device=DEVICE)
            dx.index_add_(0, took // top, s["dxs"][:kept].double())
            found.append(dx)
        return tuple(found)
    if op == "combine":
        y = torch.zeros_like(s["y"], dtype=torch.float64) if s["r"] is None else s["r"].double()
        ys, wt = s["ys"].double(), s["weights"].double()
        if case["grad"]:
            dys, dw = torch.zeros_like(ys), torch.zeros_like(wt)
        for j in range(case["top"]):
            here = torch.nonzero(s["slot"][:, j] >= 0)[:, 0]
            at = s["slot"][here, j].long()
            y[here] += wt[here, j, None] * ys[at]
            if case["grad"]:
                dy = s["dy"][here].double()
                dys[at] = wt[here, j, None] * dy
                dw[here, j] = (dy * ys[at]).sum(1)
        return (y, dys, dw) if case["grad"] else (y,)
    off = s["offsets"].tolist()
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=DEVICE)  # noqa: E731
    rows, n, k, e = s["rows"], case["n"], case["k"], case["e"]
    if op == "experts":
        y, z = new(rows, n), new(rows, n)
        for i in range(e):
            part = slice(off[i], off[i + 1])
            w = s["w"][i].double()
            z[part] = s["x"][part].double() @ (w.T if nt else w) + (0 if s["b"] is None else s["b"][i].double())
        y = _value64(z, case["act"])[0]
        return (y, z) if case["keep_z"] else (y,)
    dx, dw, db = new(rows, k), new(*s["w"].shape), new(e, n)
    for i in range(e):
        part = slice(off[i], off[i + 1])
        g = s["dy"][part].double() * _value64(s["z"][part].double(), case["act"])[1]
        w, x = s["w"][i].double(), s["x"][part].double()
        dx[part] = g @ (w if nt else w.T)
        dw[i] = g.T @ x if nt else x.T @ g
        db[i] = g.sum(0)
    return dx, dw, db
