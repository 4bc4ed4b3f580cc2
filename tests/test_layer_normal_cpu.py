"""The accuracy that csrc/layer.h states for its normal distribution function: the same steps, with the
coefficients read from the source, in exact and in float32 arithmetic, against scipy. No GPU."""
import os
import re

import numpy as np
from scipy.special import erfcx, ndtr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = np.float32


def source():
    with open(os.path.join(ROOT, "dense_gemm_tile_amd", "csrc", "layer.h")) as f:
        text = f.read()
    return text[text.index("LayerNormal layer_normal"):text.index("// GELU's tanh form")]


def number(pattern):
    return [F(v) for v in re.findall(pattern, source())]


COEFFICIENTS = number(r"float g = (-?[\d.e-]+)f") + number(r"fmaf\(g, t, (-?[\d.e-]+)f\)")


def fma(a, b, c):
    """One rounding to float32 of a b + c (the product of two float32 is exact in 64 bits)."""
    return (np.asarray(a, np.float64) * b + c).astype(F)


def phi(z):
    """layer_normal() step by step, its reciprocal and exponential rounded correctly."""
    hi_, lo_ = number(r"kHi = ([\d.e-]+)f")[0], number(r"kLo = ([\d.e-]+)f")[0]
    c = np.clip(z, F(-16), F(16))
    h = c * hi_
    hl = fma(c, lo_, fma(c, hi_, -h))
    hi = h * c
    lo = fma(hl, c, fma(h, c, -hi))
    e0 = np.exp2(-hi.astype(np.float64)).astype(F)
    e = fma(F(-0.6931471805599453) * lo, e0, e0)
    t = (1 / fma(np.abs(c), F(0.3535533905932738), F(1)).astype(np.float64)).astype(F)
    g = np.full_like(c, COEFFICIENTS[0])
    for k in COEFFICIENTS[1:]:
        g = fma(g, t, k)
    q = F(0.5) * t * g * e
    return np.where(c < 0, q, F(1) - q)


def test_the_steps_are_those_of_the_source():
    assert len(COEFFICIENTS) == 9
    for step in ("h = c * kHi, hl = __builtin_fmaf(c, kLo, __builtin_fmaf(c, kHi, -h))",
                 "hi = h * c, lo = __builtin_fmaf(hl, c, __builtin_fmaf(h, c, -hi))",
                 "__builtin_fmaf(-0.6931471805599453f * lo, e0, e0)", "0.3535533905932738f, 1.0f",
                 "0.5f * t * g * e", "c < 0.0f ? q : 1.0f - q"):
        assert step in source(), step


def test_the_polynomial():
    x = np.linspace(0, 9.4, 1000001)
    t = 1 / (1 + x / 2)
    worst = np.abs(np.polyval(np.array(COEFFICIENTS, np.float64), t) * t / erfcx(x) - 1).max()
    assert 7e-8 < worst <= 7.4e-8


def test_phi_in_float32():
    z = np.random.default_rng(0).uniform(-13, 16, 2000000).astype(F)
    worst = np.abs(phi(z) / ndtr(z.astype(np.float64)) - 1).max()
    assert 3e-7 < worst <= 4e-7
