"""Products with 4-bit weights and group scales, in float64.

Test infrastructure (see the package docstring).  Readings: two codes a byte, the even column in the low half; INT4
values are (code - zero point) times the group's scale, the zero point 8 where none is given; E2M1 is the OCP MX
4-bit element (sign, 2 exponent bits of bias 1, 1 mantissa bit; subnormals 0 and 0.5; no Inf or NaN); an E8M0 scale
code c is 2^(c - 127), 255 NaN.
"""

from __future__ import annotations

import numpy as np


def unpack_codes(w) -> np.ndarray:
    """uint8 [N, K/2] -> codes [N, K]."""
    w = np.asarray(w, dtype=np.uint8)
    return np.stack([w & 15, w >> 4], axis=-1).reshape(w.shape[0], -1)


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 1) & 3, c & 1
    v = np.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1))
    return np.where(c & 8, -v, v)


def w4_values(w, scale, fmt="int4", zero=None) -> np.ndarray:
    """[N, K] weights; scale [N, groups] as float64 values."""
    q = unpack_codes(w)
    scale = np.asarray(scale, dtype=np.float64)
    group = q.shape[1] // scale.shape[1]
    if fmt == "e2m1":
        v = e2m1_decode(q)
    else:
        z = np.full(scale.shape, 8.0) if zero is None else np.asarray(zero, dtype=np.float64)
        v = q - np.repeat(z, group, axis=1)
    return v * np.repeat(scale, group, axis=1)


def w4_gemm(x, w, scale, fmt="int4", zero=None, bias=None):
    """-> (P [M, N], S [M, N]): S = sum_k |x_k| |scale| (q + |z|) (E2M1: |q|), what the rounding errors scale with."""
    x = np.asarray(x, dtype=np.float64)
    p = x @ w4_values(w, scale, fmt, zero).T
    if bias is not None:
        p = p + np.asarray(bias, dtype=np.float64)
    a = np.abs(np.asarray(scale, dtype=np.float64))
    q = unpack_codes(w)
    group = q.shape[1] // a.shape[1]
    if fmt == "e2m1":
        big = np.abs(e2m1_decode(q))
    else:
        big = q + np.repeat(np.full(a.shape, 8.0) if zero is None else np.asarray(zero, dtype=np.float64), group, axis=1)
    return p, np.abs(x) @ (big * np.repeat(a, group, axis=1)).T
