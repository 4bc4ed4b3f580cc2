"""More layer operators that are timed: layer norms, the gate that chooses experts, products with
4-bit weights, and the output layer's cross entropy. Each has its plain form in elementary torch
operations (`own` false) and the library's calls (`own` true), on the same prepared state.

Operators and what they return:

  norm     Y = (X - mean) * rstd * gamma + beta; with `grad`, also mean, rstd, and from dY: dX (plus
           the residual stream's own gradient R where `residual`), dgamma and dbeta
  gate     logits -> the chosen experts' ids and weights; with `grad`, also the logits' gradient
           from the weights'
  w4       Y = act(X @ W' + bias) + R, W held as 4-bit codes with a scale (and a zero point) for
           each run of `group` of them
  experts  the same with one weight matrix per group of sorted rows
  loss     cross entropy of X @ W' against labels, and the log of each row's sum of exponentials;
           with `grad`, also dX and dW
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"
EPS = 1e-5


def listed():
    return [
        # The norm in front of a layer in decoding: nothing but latency.
        dict(name="norm_decode", op="norm", m=32, n=4096, dtype="bf16", grad=False, residual=False, pad=0),
        # Rows of a width that fills no piece, at an odd pitch, with float32 values.
        dict(name="norm_ragged", op="norm", m=4097, n=1033, dtype="f32", grad=True, residual=False, pad=3),
        # A training batch on a residual stream, forward and backward.
        dict(name="norm_train", op="norm", m=16384, n=4096, dtype="bf16", grad=True, residual=True, pad=0),
        # The experts of a decoding batch: latency again.
        dict(name="gate_decode", op="gate", t=32, e=64, top=4, dtype="f32", score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0, grad=False),
        # A training batch's choices among many experts in groups, balanced by a bias, and the gradient.
        dict(name="gate_train", op="gate", t=16384, e=256, top=8, dtype="f32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, grad=True),
        # One token through an output projection with 4-bit weights.
        dict(name="w4_token", op="w4", m=1, n=4096, k=4096, dtype="bf16", out="bf16", group=128, zeros=False,
             act="none", bias=False, residual=True, pad=0),
        # A batch of decoding sequences through a wide up-projection, weights with zero points.
        dict(name="w4_decode", op="w4", m=48, n=8192, k=8192, dtype="f16", out="f16", group=64, zeros=True,
             act="gelu", bias=True, residual=False, pad=0),
        # A prompt whose length and widths fill no tile.
        dict(name="w4_ragged", op="w4", m=257, n=1000, k=1032, dtype="bf16", out="f32", group=32, zeros=True,
             act="none", bias=True, residual=True, pad=3),
        # A decoding batch's choices: a few rows for each of many experts of 4-bit weights.
        dict(name="w4_experts", op="experts", t=32, top=4, e=64, n=2048, k=2048, dtype="bf16", out="bf16", group=32,
             zeros=False, act="silu", bias=False),
        # A short answer scored: the weights are read once.
        dict(name="loss_score", op="loss", t=61, v=32001, h=2048, dtype="bf16", grad=False),
        # A short training batch of a small model, a vocabulary that fills no tile.
        dict(name="loss_ragged", op="loss", t=1000, v=50001, h=1032, dtype="f16", grad=True),
        # A training batch of a large model.
        dict(name="loss_train", op="loss", t=8192, v=65536, h=4096, dtype="bf16", grad=True),
    ]


def _spread(rng, lo, hi, step=1):
    """A size of [lo, hi], spread over its logarithm, on a multiple of step where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v - v % step if v >= step else v))


def _width(rng, lo, hi):
    """A row width: mostly whole 16-byte pieces, now and then any number."""
    return _spread(rng, lo, hi, rng.choice([8, 8, 64, 128, 1]))


def draw(rng):
    op = rng.choice(["norm", "norm", "gate", "gate", "w4", "w4", "experts", "loss", "loss"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]))
    act = rng.choice(["none", "relu", "gelu", "gelu_erf", "silu"])
    if op == "norm":
        n = _width(rng, 64, 16384)
        case.update(m=_spread(rng, 1, min(16384, 16384 * 4096 // n)), n=n, grad=rng.random() < 0.6,
                    residual=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 3]))
        if rng.random() < 0.2:
            case["dtype"] = "f32"
    elif op == "gate":
        groups = rng.choice([1, 1, 1, 4, 8])
        e = groups * _spread(rng, max(1, 8 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        group_top = rng.choice([1, 2]) if e // groups > 1 else 1
        case.update(t=_spread(rng, 1, 16384), e=e, top=min(rng.choice([1, 2, 4, 6, 8]), top_groups * (e // groups)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, group_top=group_top, renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 1.0, 2.5]), grad=rng.random() < 0.5)
        if rng.random() < 0.6:
            case["dtype"] = "f32"
    elif op in ("w4", "experts"):
        case.update(group=rng.choice([32, 64, 128, 128]), zeros=rng.random() < 0.5, act=act,
                    out=rng.choice([case["dtype"], case["dtype"], "f32"]), bias=rng.random() < 0.5)
        if op == "w4":
            case.update(m=_spread(rng, 1, 512), n=_width(rng, 64, 8192), k=_width(rng, 64, 8192),
                        residual=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 3]))
        else:
            top = rng.choice([1, 2, 4, 8])
            n, k = _width(rng, 64, 4096), _width(rng, 64, 4096)
            e = max(top, min(_spread(rng, 2, 128), 64 * 4096 * 2048 // (n * k)))
            case.update(t=_spread(rng, 1, 512 // top), top=top, e=e, n=n, k=k)
    else:
        h = _width(rng, 64, 4096)
        v = _spread(rng, 1000, 65536, rng.choice([1, 8, 256]))
        case.update(t=_spread(rng, 1, 8192), v=v, h=h, grad=rng.random() < 0.6)
    return case


def _randn(gen, shape, dtype, scale=1.0, pad=0):
    """Normal values in the first shape[-1] columns of rows that are `pad` elements wider."""
    shape = list(shape)
    wide = shape[:-1] + [shape[-1] + pad]
    x = torch.randn(wide, generator=gen, device=DEVICE, dtype=torch.float32).mul_(scale).to(dtype)
    return x[..., :shape[-1]]


def _quantised(gen, shape, k, group, zeros, dtype):
    """Codes two to a byte (the lower index in the low half) of matrices [..., n][k], their scales
    and zero points."""
    runs = -(-k // group)
    codes = torch.randint(0, 256, (*shape, -(-k // 2)), generator=gen, device=DEVICE, dtype=torch.uint8)
    spread = 0.5 + torch.rand(*shape, runs, generator=gen, device=DEVICE)
    scales = (spread * (0.22 / math.sqrt(k))).to(dtype)  # codes spread 4.6 steps around their middle
    z = torch.randint(6, 11, (*shape, runs), generator=gen, device=DEVICE).to(dtype) if zeros else None
    return codes, scales, z


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, s = case["op"], dict(case)
    empty = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=DEVICE)  # noqa: E731
    if op == "norm":
        m, n, pad = case["m"], case["n"], case["pad"]
        # A residual stream: some features much larger than others, rows off centre.
        size = 0.5 + 3 * torch.rand(n, generator=gen, device=DEVICE) ** 4
        x = _randn(gen, (m, n), torch.float32) * size + 0.3 * _randn(gen, (m, 1), torch.float32)
        s["x"] = torch.nn.functional.pad(x, (0, pad)).to(dt)[:, :n]
        s["gamma"] = (1 + _randn(gen, (n,), torch.float32, 0.2)).to(dt)
        s["beta"] = _randn(gen, (n,), dt, 0.1)
        s["y"] = empty(m, n, dtype=dt)
        if case["grad"]:
            s["mean"], s["rstd"] = empty(m), empty(m)
            s["dy"] = _randn(gen, (m, n), dt, pad=pad)
            s["r"] = _randn(gen, (m, n), dt) if case["residual"] else None
            s["dx"], s["dgamma"], s["dbeta"] = empty(m, n, dtype=dt), empty(n), empty(n)
        return s
    if op == "gate":
        t, e, top = case["t"], case["e"], case["top"]
        liked = 0.5 * torch.randn(e, generator=gen, device=DEVICE)
        s["l"] = (liked + 1.5 * torch.randn(t, e, generator=gen, device=DEVICE)).to(dt)
        s["b"] = 0.1 * torch.randn(e, generator=gen, device=DEVICE) if case["bias"] else None
        s["ids"] = empty(t, top, dtype=torch.int32)
        s["weights"] = empty(t, top)
        if case["grad"]:
            s["dw"] = torch.randn(t, top, generator=gen, device=DEVICE)
            s["dl"] = empty(t, e, dtype=dt)
        return s
    if op == "loss":
        t, v, h = case["t"], case["v"], case["h"]
        s["w"] = _randn(gen, (v, h), dt, 2.0 / math.sqrt(h))
        labels = torch.randint(0, v, (t,), generator=gen, device=DEVICE)
        # Rows that know their label more or less; a few without one.
        known = 6 * torch.rand(t, 1, generator=gen, device=DEVICE)
        s["x"] = (torch.randn(t, h, generator=gen, device=DEVICE) + 0.5 * known * s["w"][labels].float()).to(dt)
        labels[torch.rand(t, generator=gen, device=DEVICE) < 0.05] = -1
        s["labels"] = labels.to(torch.int32)
        s["loss"], s["lse"] = empty(t), empty(t)
        if case["grad"]:
            # The mean over the rows with a label; float16 gradients are scaled up, as they are in training.
            size = 1024.0 if case["dtype"] == "f16" else 1.0
            s["dloss"] = torch.full((t,), size / max(1, int((labels >= 0).sum())), device=DEVICE)
            s["dx"], s["dw"] = empty(t, h, dtype=dt), empty(v, h, dtype=dt)
        return s
    n, k, out = case["n"], case["k"], DTYPES[case["out"]]
    if op == "w4":
        m, pad, shape = case["m"], case["pad"], (n,)
        s["r"] = _randn(gen, (m, n), out) if case["residual"] else None
    else:
        t, top, e = case["t"], case["top"], case["e"]
        m, pad, shape = t * top, 0, (e, n)
        ids = torch.rand(t, e, generator=gen, device=DEVICE).topk(top, dim=1).indices.reshape(-1)
        counts = torch.zeros(e, dtype=torch.int64, device=DEVICE)
        counts.index_add_(0, ids, torch.ones_like(ids))
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        s["capacity"] = int(counts.max())  # the most rows that an expert has
        s["rows"] = m
    s["x"] = _randn(gen, (m, k), dt, pad=pad)
    s["codes"], s["scales"], s["z"] = _quantised(gen, shape, k, case["group"], case["zeros"], dt)
    s["b"] = _randn(gen, shape, dt, 0.5) if case["bias"] else None
    s["y"] = empty(m, n, dtype=out)
    return s


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_norm(s):
    x, dt = s["x"].float(), s["x"].dtype
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    x = x * rstd
    gamma = s["gamma"].float()
    y = (x * gamma + s["beta"].float()).to(dt)
    if not s["grad"]:
        return (y,)
    dy = s["dy"].float()
    h = dy * gamma
    dx = rstd * (h - h.mean(1, keepdim=True) - x * (h * x).mean(1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return y, mean[:, 0], rstd[:, 0], dx.to(dt), (dy * x).sum(0), dy.sum(0)


def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_gate(s):
    # In 64 bits: which of two nearly equal experts is chosen must not hang on a rounding.
    t, e, top = s["t"], s["e"], s["top"]
    scores = _scores(s["l"].double(), s["score"])
    key = scores if s["b"] is None else scores + s["b"].double()
    if s["groups"] > 1:
        best = torch.sort(key.view(t, s["groups"], -1), dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        out = torch.ones(t, s["groups"], dtype=torch.bool, device=key.device)
        out[torch.arange(t, device=key.device)[:, None], kept] = False
        key = torch.where(out.repeat_interleave(e // s["groups"], dim=1), torch.full_like(key, -math.inf), key)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top]
    row = torch.arange(t, device=key.device)[:, None]
    w = scores[row, ids]
    total = w.sum(1, keepdim=True)
    weights = w / total if s["renorm"] else w
    found = ids.to(torch.int32), (weights * s["scale"]).float()
    if not s["grad"]:
        return found
    g = s["dw"].double() * s["scale"]
    if s["renorm"]:
        g = (g - (g * weights).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(scores)
    ds[row, ids] = g
    if s["score"] == "sigmoid":
        dl = ds * scores * (1 - scores)
    else:
        dl = scores * (ds - (ds * scores).sum(1, keepdim=True))
    return *found, dl.to(s["l"].dtype)


def _weights(s):
    """The values that the codes stand for, in float32: [..., n][k]."""
    codes, k = s["codes"], s["k"]
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)[..., :k].float()
    run = torch.arange(k, device=q.device) // s["group"]
    z = 8.0 if s["z"] is None else s["z"].float()[..., run]
    return (q - z) * s["scales"].float()[..., run]


def _plain_w4(s):
    z = s["x"].float() @ _weights(s).t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return (y.to(DTYPES[s["out"]]),)


def _plain_experts(s):
    at = torch.arange(s["rows"], device=s["x"].device)
    expert = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    place = expert * s["capacity"] + at - s["offsets"].long()[expert]
    wide = torch.zeros(s["e"] * s["capacity"], s["k"], device=s["x"].device)
    wide[place] = s["x"].float()
    z = torch.bmm(wide.view(s["e"], s["capacity"], s["k"]), _weights(s).transpose(1, 2)).view(-1, s["n"])[place]
    if s["b"] is not None:
        z = z + s["b"].float()[expert]
    return (_act(z, s["act"]).to(DTYPES[s["out"]]),)


def _plain_loss(s):
    x, w = s["x"].float(), s["w"].float()
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    row = torch.arange(s["t"], device=x.device)
    has = s["labels"] >= 0
    at = s["labels"].clamp(min=0).long()
    loss = torch.where(has, lse[:, 0] - logits[row, at], torch.zeros_like(lse[:, 0]))
    if not s["grad"]:
        return loss, lse[:, 0]
    g = torch.exp(logits - lse)
    g[row, at] -= 1
    g = g * (s["dloss"] * has)[:, None]
    return loss, lse[:, 0], (g @ w).to(s["x"].dtype), (g.t() @ x).to(s["x"].dtype)


PLAIN = {"norm": _plain_norm, "gate": _plain_gate, "w4": _plain_w4, "experts": _plain_experts, "loss": _plain_loss}


# ---------------------------------------------------------- the library's calls

def _ld(x):
    return 0 if x is None else x.stride(-2)


def _own_norm(s):
    import dense_gemm_tile_amd as dgt
    m, n, dt, x, y = s["m"], s["n"], s["dtype"], s["x"], s["y"]
    stream = torch.cuda.current_stream()
    if not s["grad"]:
        dgt.gemm_norm(m, n, dt, x, _ld(x), s["gamma"], s["beta"], EPS, y, _ld(y), None, None, stream=stream)
        return (y,)
    mean, rstd, dy, r, dx = s["mean"], s["rstd"], s["dy"], s["r"], s["dx"]
    dgt.gemm_norm(m, n, dt, x, _ld(x), s["gamma"], s["beta"], EPS, y, _ld(y), mean, rstd, stream=stream)
    size = dgt.gemm_norm_grad_workspace(m, n)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    dgt.gemm_norm_grad(m, n, dt, dy, _ld(dy), x, _ld(x), s["gamma"], mean, rstd, r, _ld(r), dx, _ld(dx), s["dgamma"],
                       s["dbeta"], ws, size, stream=stream)
    return y, mean, rstd, dx, s["dgamma"], s["dbeta"]


def _own_gate(s):
    import dense_gemm_tile_amd as dgt
    t, e, top, dt, logits = s["t"], s["e"], s["top"], s["dtype"], s["l"]
    stream = torch.cuda.current_stream()
    dgt.gemm_gate(t, e, top, dt, logits, e, s["score"], s["b"], s["groups"], s["top_groups"], s["group_top"],
                  s["renorm"], s["scale"], s["ids"], s["weights"], stream=stream)
    if not s["grad"]:
        return s["ids"], s["weights"]
    dgt.gemm_gate_grad(t, e, top, dt, logits, e, s["score"], s["renorm"], s["scale"], s["ids"], s["dw"], s["dl"], e,
                       stream=stream)
    return s["ids"], s["weights"], s["dl"]


def _own_w4(s):
    import dense_gemm_tile_amd as dgt
    x, c, sc, r, y = s["x"], s["codes"], s["scales"], s["r"], s["y"]
    dgt.gemm_linear_w4(s["m"], s["n"], s["k"], s["dtype"], x, _ld(x), c, 2 * _ld(c), sc, s["z"], _ld(sc), s["group"],
                       s["b"], s["act"], r, _ld(r), y, _ld(y), s["out"], stream=torch.cuda.current_stream())
    return (y,)


def _own_experts(s):
    import dense_gemm_tile_amd as dgt
    x, c, sc, y = s["x"], s["codes"], s["scales"], s["y"]
    dgt.gemm_grouped_w4(s["e"], s["rows"], s["n"], s["k"], s["dtype"], s["offsets"], x, _ld(x), c, 2 * _ld(c),
                        2 * c.stride(0), sc, s["z"], _ld(sc), sc.stride(0), s["group"], s["b"], s["act"], None, 0, y,
                        _ld(y), s["out"], stream=torch.cuda.current_stream())
    return (y,)


def _own_loss(s):
    import dense_gemm_tile_amd as dgt
    t, v, h, dt, x, w = s["t"], s["v"], s["h"], s["dtype"], s["x"], s["w"]
    stream = torch.cuda.current_stream()
    size = dgt.gemm_loss_workspace(t, v, h)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    dgt.gemm_loss(t, v, h, dt, x, _ld(x), w, _ld(w), s["labels"], s["loss"], s["lse"], ws, size, stream=stream)
    if not s["grad"]:
        return s["loss"], s["lse"]
    dx, dw = s["dx"], s["dw"]
    size = dgt.gemm_loss_grad_workspace(t, v, h)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    dgt.gemm_loss_grad(t, v, h, dt, x, _ld(x), w, _ld(w), s["labels"], s["lse"], s["dloss"], dx, _ld(dx), dw, _ld(dw),
                       dt, False, ws, size, stream=stream)
    return s["loss"], s["lse"], dx, dw


OWN = {"norm": _own_norm, "gate": _own_gate, "w4": _own_w4, "experts": _own_experts, "loss": _own_loss}


# ------------------------------------------------------------ work and definition

def work(case):
    """Bytes (each input read once, each output written once) and operations of one pass."""
    size = {"f16": 2, "bf16": 2, "f32": 4}
    d, op, grad = size[case["dtype"]], case["op"], case.get("grad", False)
    if op == "norm":
        m, n = case["m"], case["n"]
        return {"bytes": d * (m * n * (2 + grad * (2 + case["residual"])) + 2 * n) + grad * 8 * (m + n),
                "flops": m * n * (8 + 14 * grad)}
    if op == "gate":
        t, e, top = case["t"], case["e"], case["top"]
        return {"bytes": t * (d * e * (1 + grad) + top * (8 + 4 * grad)) + 4 * e * case["bias"],
                "flops": t * e * (4 + 6 * grad)}
    if op == "loss":
        t, v, h = case["t"], case["v"], case["h"]
        return {"bytes": d * h * (t + v) + 12 * t + grad * (4 * t + d * h * (t + v)),
                "flops": (6 if grad else 2) * t * v * h}
    n, k, o = case["n"], case["k"], size[case["out"]]
    runs = -(-k // case["group"])
    one = n * (-(-k // 2) + d * runs * (1 + case["zeros"]) + d * case["bias"])
    if op == "w4":
        m = case["m"]
        return {"bytes": one + d * m * k + o * m * n * (1 + case["residual"]), "flops": 2 * m * n * k}
    rows, e = case["t"] * case["top"], case["e"]
    used = e * (1 - (1 - 1 / e) ** rows)  # experts that get a row, were all liked alike
    return {"bytes": int(used * one + d * rows * k + o * rows * n + 4 * (e + 1)), "flops": 2 * rows * n * k}


def _value64(z, act):
    """The activation, from its definition, in 64 bits."""
    if act == "relu":
        return torch.maximum(z, 0 * z)
    if act == "gelu":  # z * sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3))
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "gelu_erf":
        return z * torch.special.ndtr(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _exact_gate(case, s):
    t, e, per = case["t"], case["e"], case["e"] // case["groups"]
    logits = s["l"].double().requires_grad_(True)
    p = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)
    key = p.detach() + (0 if s["b"] is None else s["b"].double())
    # An item's rank: the items that come before it, counted by comparisons.
    before = torch.ones(e, e, dtype=torch.bool, device=DEVICE).tril(-1)  # [i, j]: j < i

    def ranks(v):
        n = v.shape[1]
        found = []
        for part in v.split(max(1, (1 << 26) // (n * n))):
            a, b = part[:, :, None], part[:, None, :]
            found.append(((b > a) | ((b == a) & before[:n, :n])).sum(2))
        return torch.cat(found)
    if case["groups"] > 1:
        by = key.view(t, case["groups"], per)
        best = by.topk(case["group_top"], dim=2).values.sum(2)
        kept = ranks(best) < case["top_groups"]
        key = torch.where(kept[:, :, None], by, torch.full_like(by, -math.inf)).view(t, e)
    rank = ranks(key)
    ids = torch.stack([(rank == j).to(torch.int8).argmax(1) for j in range(case["top"])], 1)
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    found = [ids.to(torch.int32), w.detach()]
    if case["grad"]:
        found.append(torch.autograd.grad(w, logits, s["dw"].double())[0])
    return tuple(found)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(case, s)
    if op == "norm":
        x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + EPS).rsqrt()
        unit = (x - mean[:, None]) * rstd[:, None]
        y = unit * gamma + beta
        if not case["grad"]:
            return (y,)
        dy, n = s["dy"].double(), case["n"]
        h = dy * gamma
        dx = (n * h - h.sum(1)[:, None] - unit * (unit * h).sum(1)[:, None]) * (rstd / n)[:, None]
        if s["r"] is not None:
            dx += s["r"]
        return y, mean, rstd, dx, torch.einsum("mn,mn->n", dy, unit), dy.sum(0)
    if op == "loss":
        # Pieces of rows, so that the logits of a large case are not held at once.
        x, w, has = s["x"].double(), s["w"].double(), s["labels"] >= 0
        loss, lse = torch.zeros(case["t"], dtype=torch.float64, device=DEVICE), []
        dx, dw = [], torch.zeros_like(w) if case["grad"] else None
        for lo in range(0, case["t"], 1024):
            part = slice(lo, lo + 1024)
            logits = x[part] @ w.T
            lse.append(torch.logsumexp(logits, 1))
            rows = torch.nonzero(has[part])[:, 0]
            at = s["labels"][part][rows].long()
            loss[lo + rows] = lse[-1][rows] - logits[rows, at]
            if case["grad"]:
                p = torch.softmax(logits, 1)
                p[rows, at] -= 1
                p *= (s["dloss"][part].double() * has[part])[:, None]
                dx.append(p @ w)
                dw += p.T @ x[part]
        return (loss, torch.cat(lse), torch.cat(dx), dw) if case["grad"] else (loss, torch.cat(lse))

    def values(codes, scales, z):
        q = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=DEVICE)
        q[:, 0::2], q[:, 1::2] = (codes % 16).double(), (codes // 16).double()
        for j in range(scales.shape[1]):
            part = q[:, j * case["group"]:(j + 1) * case["group"]]
            part -= 8 if z is None else z[:, j, None].double()
            part *= scales[:, j, None].double()
        return q[:, :case["k"]]
    x = s["x"].double()
    if op == "w4":
        z = x @ values(s["codes"], s["scales"], s["z"]).T + (0 if s["b"] is None else s["b"].double())
        return (_value64(z, case["act"]) + (0 if s["r"] is None else s["r"].double()),)
    off = s["offsets"].tolist()
    z = torch.zeros(s["rows"], case["n"], dtype=torch.float64, device=DEVICE)
    for i in range(case["e"]):
        part = slice(off[i], off[i + 1])
        w = values(s["codes"][i], s["scales"][i], None if s["z"] is None else s["z"][i])
        z[part] = x[part] @ w.T + (0 if s["b"] is None else s["b"][i].double())
    return (_value64(z, case["act"]),)
