"""Shared by the tests of the layer operators: seeded inputs, plain definitions in 64 bits, and
the tolerances that the arithmetic implies."""
from __future__ import annotations

import math

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "gelu_erf", "silu"]
U32 = 2.0 ** -24  # half a step of float32, relative
DEV = "cuda:0"


def half_step(dtype: str) -> float:
    return torch.finfo(DT[dtype]).eps / 2


def act64(z: torch.Tensor, act: str) -> torch.Tensor:
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "gelu_erf":
        return z * torch.special.ndtr(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z: torch.Tensor, act: str) -> torch.Tensor:
    z = z.detach().clone().requires_grad_(True)
    return torch.autograd.grad(act64(z, act).sum(), z)[0]


def randn(gen, *shape, dtype="f32", scale=1.0, pad=0, fill=float("nan")):
    """Seeded values on the device in rows `pad` elements wider, the padding filled."""
    x = torch.full((*shape[:-1], shape[-1] + pad), fill, dtype=DT[dtype])
    x[..., :shape[-1]] = (torch.randn(*shape, generator=gen) * scale).to(DT[dtype])
    return x.to(DEV)[..., :shape[-1]]


def ld(x):
    return 0 if x is None else x.stride(-2)


def out(*shape, dtype="f32", pad=0):
    """An output whose every element, padding too, holds NaN."""
    return torch.full((*shape[:-1], shape[-1] + pad), float("nan"), dtype=DT[dtype],
                      device=DEV)[..., :shape[-1]]


def padding_untouched(x: torch.Tensor) -> bool:
    wide = torch.as_strided(x, (*x.shape[:-1], x.stride(-2)), x.stride(), x.storage_offset()) \
        if x.stride(-2) > x.shape[-1] else None
    return wide is None or bool(torch.isnan(wide[..., x.shape[-1]:]).all())


def close(got: torch.Tensor, want: torch.Tensor, tol: torch.Tensor, what=""):
    """|got - want| <= tol elementwise, in 64 bits; NaN and infinities have to be the same."""
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    bad = torch.where(fine, ~((got - want).abs() <= tol), ~same)
    if bool(bad.any()):
        i = tuple(torch.nonzero(bad)[0].tolist())
        t = tol[i] if isinstance(tol, torch.Tensor) and tol.dim() else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()} wanted {want[i].item()} within {float(t):.3g}")


def sum_tol(n: int, sums: torch.Tensor) -> torch.Tensor:
    """How far a float32 sum of n products may be off, in any order: n roundings of partial sums,
    each at most half a step of the sum of absolute values (`sums`)."""
    return (n + 2) * U32 * sums


# An activation's value and slope come from a few float32 operations on z: exp of a number of
# at most about 100 carries that many half steps relative, the rest a handful.
ACT_STEPS = 128


def tiny(dtype: str) -> float:
    """Half the distance between the smallest numbers of a type."""
    return torch.finfo(DT[dtype]).tiny * torch.finfo(DT[dtype]).eps / 2


def linear_want(x, w, b, r, act, dtype, out_dtype):
    """Y, Z and their tolerances from operands already in op() order: x [M,K], w [K,N]."""
    x, w = x.double(), w.double()
    z, mag = x @ w, x.abs() @ w.abs()
    if b is not None:
        z, mag = z + b.double(), mag + b.double().abs()
    y = act64(z, act)
    off = sum_tol(x.shape[1] + 1, mag)
    ytol = 1.2 * off + ACT_STEPS * U32 * y.abs()  # no slope here passes 1.2
    if r is not None:
        y = y + r.double()
        ytol = ytol + U32 * y.abs()
    ytol = ytol * (1 + half_step(out_dtype)) + half_step(out_dtype) * y.abs() + tiny(out_dtype)
    ztol = off * (1 + half_step(dtype)) + half_step(dtype) * z.abs() + tiny(dtype)
    return y, z, ytol, ztol


def offsets_of(sizes):
    o = [0]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int32, device=DEV)
