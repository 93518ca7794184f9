"""Fit the polynomial of the kernels' FMA-pipe score cap (``kTanhC*`` of
score_mod.cuh).

For |u| <= kTanhMax, tanh(u) = u * g(u^2) with g(w) = tanh(sqrt w) / sqrt w,
which is smooth at 0.  g is approximated on [0, kTanhMax^2] by a polynomial in
w whose coefficients minimise the maximum RELATIVE error (the Remez exchange
algorithm, weighted by 1 / g), so that small scores keep their relative
accuracy.  Degree 5 on [0, 1] errs by 5.9e-7, about as much as the
special-function path (2^-21 of the cap); the kernel takes that path where a score of the
tile lies outside.

    python context_blocks_b200/csrc/gen_tanh_poly.py
"""

import numpy as np


def g(w):
    u = np.sqrt(np.asarray(w, dtype=np.float64))
    small = u < 1e-4
    return np.where(small, 1.0 - u * u / 3.0, np.tanh(np.where(small, 1.0, u)) / np.where(small, 1.0, u))


def fit(degree: int = 5, umax: float = 1.0, iters: int = 40):
    """Coefficients c_0..c_degree (float64) of the polynomial in w and its max
    relative error on [0, umax^2]."""
    m = degree + 2
    top = umax * umax
    ref = top * 0.5 * (1.0 - np.cos(np.pi * np.arange(m) / (m - 1)))
    grid = np.linspace(0.0, top, 200001)
    gg = g(grid)
    c = None
    for _ in range(iters):
        y = g(ref)
        a = np.hstack([np.vander(ref, degree + 1, increasing=True), (-(-1.0) ** np.arange(m) * y)[:, None]])
        c = np.linalg.solve(a, y)[:-1]
        err = (np.vander(grid, degree + 1, increasing=True) @ c - gg) / gg
        flips = np.nonzero(np.sign(err[1:]) != np.sign(err[:-1]))[0]
        bounds = np.concatenate([[0], flips + 1, [len(grid)]])
        ext = [lo + int(np.argmax(np.abs(err[lo:hi]))) for lo, hi in zip(bounds[:-1], bounds[1:])]
        if len(ext) != m:
            break
        new_ref = grid[ext]
        if np.allclose(new_ref, ref, atol=1e-12, rtol=0):
            break
        ref = new_ref
    err = (np.vander(grid, degree + 1, increasing=True) @ c - gg) / gg
    return c, float(np.max(np.abs(err)))


def simulate(c32: np.ndarray, u: np.ndarray) -> np.ndarray:
    """The kernel's float32 steps for u = s * k: w = u * u, Horner with fused
    steps (taken in float64 and rounded once each), then u * p(w)."""
    u = np.asarray(u, dtype=np.float32)
    w = (u * u).astype(np.float32)
    p = np.full_like(u, c32[-1])
    for k in range(len(c32) - 2, -1, -1):
        p = (p.astype(np.float64) * w + np.float64(c32[k])).astype(np.float32)
    return (u * p).astype(np.float32)


if __name__ == "__main__":
    for degree in (4, 5, 6):
        c, e = fit(degree)
        print(f"degree {degree}:", ", ".join(f"{v:.9e}f" for v in c.astype(np.float32)), f" max relative error {e:.3e}")
        u = np.linspace(-1.0, 1.0, 400002)
        r = simulate(c.astype(np.float32), u).astype(np.float64)
        print(f"  float32 steps: {np.max(np.abs(r - np.tanh(u)) / np.abs(np.tanh(u))):.3e}")
