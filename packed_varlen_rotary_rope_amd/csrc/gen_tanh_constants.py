"""Generate tanh_constants.h: the fp32 polynomial with which the attention kernels cap scores,
each coefficient rounded once from a 60-digit mpmath value.

For |y| <= NEAR, tanh(y) = y P(y^2) with P a Chebyshev fit of degree DEGREE on [0, NEAR^2]
(mpmath.chebyfit). Its error with fp32 coefficients, evaluated by Horner's rule in fp32 as
the kernels do, is checked below MOST relative before the header is written; above NEAR the
kernels take 1 - 2 / (1 + exp(2 |y|)), which loses about a bit there.

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


def text():
    c = coefficients()
    error = worst(c)
    if not error < MOST:
        raise SystemExit(f"the fit is off by {error:.3g}")
    lines = ["// Generated by gen_tanh_constants.py -- do not edit. tanh(y) = y sum_i kTanhPoly[i] y^(2 i)",
             f"// for |y| <= kTanhNear, relative error {error:.1e} as evaluated in fp32.", "#pragma once", "",
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
