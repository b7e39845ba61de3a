"""Layer norm and RMS norm, forward and backward, in float64.

Test infrastructure (see the package docstring).  Definitions:

* mean = sum_c s / n (RMS norm: 0), var = sum_c (s - mean)^2 / n,
  rstd = 1 / sqrt(var + eps), y = (s - mean) rstd gamma + beta.
* Backward, from the chain rule: with xh = (x - mean) rstd and g = dy gamma,
  dx = rstd (g - mean_c(g) - xh mean_c(g xh)) (RMS norm: without mean_c(g)),
  dgamma = sum_r dy xh, dbeta = sum_r dy.  The derivation is pinned by
  differences of the forward in tests/test_oracle_norm.py.
"""

from __future__ import annotations

import numpy as np


def norm_forward(s, gamma, beta=None, eps=1e-5, kind="layer"):
    """-> (y, mean, rstd); s [rows, cols] float64."""
    s = np.asarray(s, dtype=np.float64)
    mean = s.mean(axis=1) if kind == "layer" else np.zeros(s.shape[0])
    centered = s - mean[:, None]
    with np.errstate(divide="ignore"):
        rstd = 1.0 / np.sqrt((centered * centered).mean(axis=1) + eps)
    y = centered * rstd[:, None] * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, mean, rstd


def norm_backward(dy, x, gamma, mean, rstd, kind="layer", dskip=None):
    """-> (dx, dgamma, dbeta), the statistics taken as given."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    rstd = np.asarray(rstd, dtype=np.float64)[:, None]
    xh = (x - np.asarray(mean, dtype=np.float64)[:, None] if kind == "layer" else x) * rstd
    g = dy * np.asarray(gamma, dtype=np.float64)
    inner = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        inner = inner - g.mean(axis=1, keepdims=True)
    dx = rstd * inner
    if dskip is not None:
        dx = dx + np.asarray(dskip, dtype=np.float64)
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)
