"""Derive the polynomial coefficients the softmax kernels evaluate on the FMA pipe.

Method: Remez exchange for the minimax *relative* error.
  tanh_poly.h  q(v) ~ tanh(u) / u with v = u^2, u in [0, U], so that
               tanh(u) = u q(u^2) is odd by construction.
  tanh2_poly.h the same on the narrower range |u| <= 1/2 at degree 2.
  tanh_fine_poly.h the same on |u| <= 3/4, the error a tenth.
Run: ``python gen_poly.py``; writes the headers next to this file.
"""
from __future__ import annotations

import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
TANH_RANGE = 1.0       # |u| <= U on the polynomial; beyond it the kernels use 1 - 2 / (e^{2u} + 1)
TANH_DEGREE = 4        # degree in v = u^2 (u^9)
# A cheaper tier for small arguments: where every |u| of a warp's tile half is
# <= 1/2 (soft-cap workloads whose scores stay well inside the cap), degree 2
# reaches about the same error as degree 4 on |u| <= 1.
TANH2_RANGE = 0.5
TANH2_DEGREE = 2
# The paged kernels' polynomial: a cap far above the scores is one of their
# inputs, and the polynomial's relative error is then that of the scores.
TANH_FINE_RANGE = 0.75
TANH_FINE_DEGREE = 4


def remez(func, lo, hi, deg, iters=60, grid_n=200001):
    """Minimax relative-error polynomial c[0] + c[1] x + ... for func on [lo, hi]."""
    n = deg + 2
    k = np.arange(n)
    x = 0.5 * (lo + hi) + 0.5 * (hi - lo) * np.cos(np.pi * (n - 1 - k) / (n - 1))
    grid = np.linspace(lo, hi, grid_n)
    for _ in range(iters):
        g = func(x)
        A = np.zeros((n, n))
        for j in range(deg + 1):
            A[:, j] = x ** j
        A[:, deg + 1] = ((-1.0) ** k) * g
        sol = np.linalg.solve(A, g)
        c = sol[:deg + 1]
        err = (np.polyval(c[::-1], grid) - func(grid)) / func(grid)
        s = np.sign(err)
        s[s == 0] = 1
        segs = np.split(np.arange(grid.size), np.flatnonzero(np.diff(s)) + 1)
        ext = np.array([seg[np.argmax(np.abs(err[seg]))] for seg in segs])
        if ext.size < n:
            break
        while ext.size > n:
            ext = ext[1:] if abs(err[ext[0]]) < abs(err[ext[-1]]) else ext[:-1]
        x = grid[ext]
    err = (np.polyval(c[::-1], grid) - func(grid)) / func(grid)
    return c, float(np.abs(err).max())


def tanh_over_u(v):
    u = np.sqrt(np.maximum(v, 0.0))
    out = np.ones_like(u)
    nz = u > 1e-12
    out[nz] = np.tanh(u[nz]) / u[nz]
    return out


def tanh_coeffs(deg=TANH_DEGREE, U=TANH_RANGE):
    return remez(tanh_over_u, 0.0, U * U, deg)


def _write(path, title, names, c, extra):
    lines = [f"// {os.path.basename(path)} -- generated by gen_poly.py ({title}).  Do not edit.",
             "#pragma once", "namespace fa {"]
    for i, v in enumerate(c):
        lines.append(f"constexpr float {names}{i} = {float(np.float32(v))!r}f;")
    lines += extra + ["}  // namespace fa"]
    with open(path, "w") as f:
        f.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    c, e = tanh_coeffs()
    _write(os.path.join(HERE, "tanh_poly.h"),
           f"Remez minimax of tanh(u)/u in v = u^2, |u| <= {TANH_RANGE}, degree {TANH_DEGREE} in v, "
           f"max relative error {e:.3e}",
           "kTanhC", c, [f"constexpr int kTanhDegree = {TANH_DEGREE};",
                         f"constexpr float kTanhRange = {TANH_RANGE}f;",
                         f"constexpr float kTanhMaxRelErr = {e:.3e}f;"])
    print(f"tanh: {c.tolist()} max rel err {e:.3e}")
    c, e = tanh_coeffs(TANH2_DEGREE, TANH2_RANGE)
    _write(os.path.join(HERE, "tanh2_poly.h"),
           f"Remez minimax of tanh(u)/u in v = u^2, |u| <= {TANH2_RANGE}, degree {TANH2_DEGREE} in v, "
           f"max relative error {e:.3e}",
           "kTanh2C", c, [f"constexpr int kTanh2Degree = {TANH2_DEGREE};",
                          f"constexpr float kTanh2Range = {TANH2_RANGE}f;",
                          f"constexpr float kTanh2MaxRelErr = {e:.3e}f;"])
    print(f"tanh2: {c.tolist()} max rel err {e:.3e}")
    c, e = tanh_coeffs(TANH_FINE_DEGREE, TANH_FINE_RANGE)
    _write(os.path.join(HERE, "tanh_fine_poly.h"),
           f"Remez minimax of tanh(u)/u in v = u^2, |u| <= {TANH_FINE_RANGE}, degree {TANH_FINE_DEGREE} in v, "
           f"max relative error {e:.3e}",
           "kTanhFineC", c, [f"constexpr float kTanhFineRange = {TANH_FINE_RANGE}f;"])
    print(f"tanh fine: {c.tolist()} max rel err {e:.3e}")
