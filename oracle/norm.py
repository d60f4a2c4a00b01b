"""fp64 oracle of the root-mean-square norm of a pre-norm block and its
gradient: the formulas and nothing else.

  r = x + resid,  c = (mean_j r_j^2 + eps)^(-1/2),  u_j = r_j c w_j
"""
from __future__ import annotations

import numpy as np


def rmsnorm(x, resid, w, eps):
    """(r, c, u) of x [T, d], resid [T, d] or None, w [d]."""
    r = np.asarray(x, np.float64) if resid is None else np.asarray(x, np.float64) + np.asarray(resid, np.float64)
    c = 1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)
    return r, c, r * c[:, None] * np.asarray(w, np.float64)


def rmsnorm_backward(du, r, w, c, dr=None):
    """(dx, dw) for dL/du = du, with c [T] the forward's; dr: gradient that
    reaches r by another way."""
    du, r, w, c = (np.asarray(a, np.float64) for a in (du, r, w, c))
    xhat = r * c[:, None]
    g = du * w
    dx = c[:, None] * (g - xhat * np.mean(g * xhat, axis=1, keepdims=True))
    if dr is not None:
        dx = dx + np.asarray(dr, np.float64)
    return dx, np.sum(du * xhat, axis=0)
