"""fp64 oracle of the gated residual update with the norms around it (NumPy)."""

from __future__ import annotations

import numpy as np

from .score_mod import _f64


def normed(v, kind, eps):
    if kind == "layer":
        return (v - v.mean(-1, keepdims=True)) / np.sqrt(v.var(-1, keepdims=True) + eps)
    if kind == "rms":
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v


def gate_residual_norm(y, x, gate=None, post="none", post_weight=None, norm="rms", norm_weight=None, scale=None,
                       shift=None, residual_scale=1.0, eps=1e-6):
    """(x_new, h) in fp64; h is None without a norm."""
    t = normed(_f64(y), post, eps)
    if post_weight is not None:
        t = t * _f64(post_weight)
    if gate is not None:
        t = t * _f64(gate)[:, None]
    x = residual_scale * _f64(x) + t
    if norm == "none":
        return x, None
    h = normed(x, norm, eps)
    if norm_weight is not None:
        h = h * _f64(norm_weight)
    if scale is not None:
        h = h * (1.0 + _f64(scale)[:, None])
    if shift is not None:
        h = h + _f64(shift)[:, None]
    return x, h
