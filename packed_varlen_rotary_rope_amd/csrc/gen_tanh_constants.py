"""Generate tanh_constants.h: the fp32 polynomial with which the attention kernels cap scores,
each coefficient rounded once from a 60-digit mpmath value.

For |y| <= NEAR, tanh(y) = y P(y^2) with P a Chebyshev fit of degree DEGREE on [0, NEAR^2]
(mpmath.chebyfit). Its error with fp32 coefficients, evaluated by Horner's rule in fp32 as
the kernels do, is checked below MOST relative before the header is written; above NEAR the
kernels take 1 - 2 / (1 + exp(2 |y|)), which loses about a bit there. That form is checked below
MOST with exp2 and the reciprocal rounded to nearest, and below MOST_BY_STEPS with either a step off
in the direction that hurts, which the instructions' specification leaves open (none of all fp32
arguments, run on gfx950, is off by more than 1.85e-7).

Usage: python -m packed_varlen_rotary_rope_amd.csrc.gen_tanh_constants [--check]
(--check: exit 1 if the committed header differs from a fresh generation).
"""
from __future__ import annotations

import os
import sys

import mpmath as mp
import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
OUT = os.path.join(HERE, "tanh_constants.h")
DEGREE = 4
NEAR = mp.mpf("0.6")
MOST = 2.0 ** -22
MOST_BY_STEPS = 2.0 ** -21.7
mp.mp.dps = 60


def ratio(z):
    """tanh(y) / y at z = y^2."""
    y = mp.sqrt(z)
    return mp.tanh(y) / y if z > mp.mpf(10) ** -40 else 1 - z / 3


def coefficients():
    return [np.float32(str(c)) for c in mp.chebyfit(ratio, [0, NEAR ** 2], DEGREE + 1)][::-1]


def evaluate(c, y):
    """The kernels' evaluation: Horner with fused multiply-adds in fp32."""
    y = np.float32(y)
    z = np.float32(y * y)
    x = c[-1]
    for a in c[-2::-1]:  # a product of two floats and the sum are exact enough in 64 bits
        x = np.float32(np.float64(x) * np.float64(z) + np.float64(a))
    return np.float32(y * x)


def worst(c):
    out = 0.0
    near = float(NEAR)
    for y in np.concatenate([np.linspace(2.0 ** -20, near, 4001), near * 2.0 ** np.linspace(-100, 0, 501)]):
        exact = mp.tanh(mp.mpf(float(np.float32(y))))
        out = max(out, float(abs(mp.mpf(float(evaluate(c, y))) / exact - 1)))
    return out


def worst_far(steps):
    """The error of 1 - 2 / (1 + exp2(2 log2 e y)) as the kernels form it in fp32, exp2 and the reciprocal
    off by `steps` of their last place, at every fp32 y from NEAR to 2 (it falls from there on)."""
    first = np.float32(str(NEAR)).view(np.int32)
    y = np.arange(first + 1, np.float32(2).view(np.int32) + 1, dtype=np.int32).view(np.float32)
    up = np.float32(np.copysign(np.inf, steps))

    def off(x, towards):
        return np.nextafter(x, towards) if steps else x

    e = off(np.exp2((y * np.float32(str(2 / mp.log(2)))).astype(np.float64)).astype(np.float32), up)
    r = off(np.float32(1) / (np.float32(1) + e), -up)  # a larger e makes it smaller
    t = (1.0 - 2.0 * r.astype(np.float64)).astype(np.float32)
    return float(np.abs(t / np.tanh(y.astype(np.float64)) - 1).max())


def text():
    c = coefficients()
    error, far, stepped = worst(c), worst_far(0), max(worst_far(1), worst_far(-1))
    if not (error < MOST and far < MOST and stepped < MOST_BY_STEPS):
        raise SystemExit(f"off by {error:.3g} up to {float(NEAR)}, {far:.3g} and {stepped:.3g} beyond")
    lines = ["// Generated by gen_tanh_constants.py -- do not edit. tanh(y) = y sum_i kTanhPoly[i] y^(2 i)",
             f"// for |y| <= kTanhNear, relative error {error:.1e} as evaluated in fp32; beyond it 1 - 2 / (1 + exp(2 |y|)),",
             f"// {far:.1e} with exp2 and the reciprocal rounded to nearest, {stepped:.1e} with either off by a step.",
             "#pragma once", "",
             "namespace attn {", "", f"constexpr float kTanhNear = {float(np.float32(str(NEAR))):.9e}f;",
             f"constexpr int kTanhDegree = {DEGREE};",
             f"constexpr float kTanhPoly[{DEGREE + 1}] = {{" + ", ".join(f"{float(x):.9e}f" for x in c) + "};",
             "", "}  // namespace attn", ""]
    return "\n".join(lines)


def main():
    fresh = text()
    if "--check" in sys.argv:
        sys.exit(0 if open(OUT).read() == fresh else 1)
    with open(OUT, "w") as f:
        f.write(fresh)


if __name__ == "__main__":
    main()
