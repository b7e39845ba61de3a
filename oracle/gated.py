"""The gated feed-forward block, forward and backward, in float64.

Test infrastructure (see the package docstring).  Definitions:

* P = A B^T + bias with B = [gate rows; up rows]; D = act(P[:, :N]) * P[:, N:].
* act is silu(x) = x / (1 + exp(-x)), or the tanh form of GELU (oracle.gemm).
* Backward, by the product and chain rules: for the gradient dh of D,
  dgate = dh up act'(gate), dup = dh act(gate).
"""

from __future__ import annotations

import numpy as np

from .gemm import dgelu_tanh, gelu_tanh

ACTIVATIONS = ("silu", "gelu")


def activation(x, act: str) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    if act == "gelu":
        return gelu_tanh(x)
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def activation_grad(x, act: str) -> np.ndarray:
    """act'(x); silu: with s = 1 / (1 + exp(-x)), (x s)' = s + x s (1 - s)."""
    x = np.asarray(x, dtype=np.float64)
    if act == "gelu":
        return dgelu_tanh(x)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-x))
    return s + x * s * (1.0 - s)


def gated(p, act: str) -> np.ndarray:
    """act(gate) * up of the pre-activations p [M, 2N] = [gate | up]."""
    gate, up = np.split(np.asarray(p, dtype=np.float64), 2, axis=1)
    return activation(gate, act) * up


def gated_grad(dh, p, act: str) -> np.ndarray:
    """[dgate | dup] for the gradient dh [M, N] of gated(p)."""
    gate, up = np.split(np.asarray(p, dtype=np.float64), 2, axis=1)
    dh = np.asarray(dh, dtype=np.float64)
    return np.concatenate([dh * up * activation_grad(gate, act), dh * activation(gate, act)], axis=1)
