"""The router of a mixture-of-experts block, the sort of its slots, and the rows' way to the experts and back, in float64
and exact integers.

Test infrastructure (see the package docstring).  Definitions:

* s = softmax(l) over the experts whose logit is not -inf, or 1 / (1 + exp(-l)); the chosen experts are the topk of
  the largest s + bias (l without a bias), equal ones in rising order; -1 where none is left.
* w_k = scale s_k / S, S the sum of the chosen scores, or 1.
* A slot t topk + k names one expert of token t; rows are the slots in the order (expert, slot).
* dispatch: y[row] = x[token of the row's slot]; combine: y[t] = sum_k w[t, k] rows[row of (t, k)].
* Backward, by the chain rule: see the functions.  The derivations are pinned by differences of the forward in
  tests/test_oracle_moe.py.
"""

from __future__ import annotations

import numpy as np


def scores(logits, score: str) -> np.ndarray:
    x = np.asarray(logits, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = np.nanmax(x, axis=1, keepdims=True, initial=-np.inf)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total == 0, 1.0, total)


def route(logits, topk: int, score="softmax", bias=None, normalize=True, scale=1.0):
    """-> (experts int32 [T, topk], weights [T, topk])."""
    x = np.asarray(logits, dtype=np.float64)
    s = scores(x, score)
    key = x if bias is None else np.where(np.isneginf(x), -np.inf, s + np.asarray(bias, dtype=np.float64))
    key = np.where(np.isnan(key), -np.inf, key)
    order = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    live = np.take_along_axis(key, order, 1) > -np.inf
    experts = np.where(live, order, -1).astype(np.int32)
    return experts, scale * shares(s, experts, normalize)


def shares(s, experts, normalize=True) -> np.ndarray:
    """The scores of given experts (-1: 0), divided by their sum with normalize."""
    live = experts >= 0
    w = np.where(live, np.take_along_axis(s, np.where(live, experts, 0), 1), 0.0)
    if normalize:
        # in the log domain's stead: tests of scores too small for float64 have their logarithms
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total == 0, 1.0, total)
    return w


def route_backward(logits, experts, dweights, score="softmax", normalize=True, scale=1.0) -> np.ndarray:
    """dlogits [T, E].  With g_k = scale dw_k and w_k = s_k / S: dL/ds_k = (g_k - sum_j g_j w_j) / S (normalize), g_k
    (not); softmax: dl_e = s_e (ds_e - sum_j ds_j s_j); sigmoid: dl_e = ds_e s_e (1 - s_e)."""
    x = np.asarray(logits, dtype=np.float64)
    s = scores(x, score)
    live = (experts >= 0) & (experts < x.shape[1])
    at = np.where(live, experts, 0)
    g = np.where(live, scale * np.asarray(dweights, dtype=np.float64), 0.0)
    sk = np.where(live, np.take_along_axis(s, at, 1), 0.0)
    if normalize:
        S = sk.sum(axis=1, keepdims=True)
        S = np.where(S == 0, 1.0, S)
        g = np.where(live, (g - (g * sk).sum(axis=1, keepdims=True) / S) / S, 0.0)
    ds = np.zeros_like(s)
    for k in range(experts.shape[1]):
        t = np.nonzero(live[:, k])[0]
        ds[t, experts[t, k]] += g[t, k]
    if score == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))


def sort_slots(experts, num_experts: int):
    """-> (m_splits [num_experts], row_of [slots], slot_of [slots]), int32."""
    flat = np.asarray(experts).reshape(-1)
    slots = [np.nonzero(flat == e)[0] for e in range(num_experts)]
    m_splits = np.array([len(s) for s in slots], dtype=np.int32)
    order = np.concatenate(slots) if slots else np.zeros(0, dtype=np.int64)
    row_of = np.full(flat.size, -1, dtype=np.int32)
    row_of[order] = np.arange(order.size)
    slot_of = np.full(flat.size, -1, dtype=np.int32)
    slot_of[:order.size] = order
    return m_splits, row_of, slot_of


def combine(rows, row_of, weights=None) -> np.ndarray:
    """[T, cols] of rows [R, cols], row_of [T, topk]; weights None: 1."""
    rows = np.asarray(rows, dtype=np.float64)
    live = (row_of >= 0) & (row_of < rows.shape[0])
    y = np.zeros((row_of.shape[0], rows.shape[1]))
    for k in range(row_of.shape[1]):
        t = np.nonzero(live[:, k])[0]
        w = 1.0 if weights is None else np.asarray(weights, dtype=np.float64)[t, k, None]
        y[t] += w * rows[row_of[t, k]]
    return y


def combine_backward(dy, rows, row_of, weights):
    """-> (drows [R, cols], zeros where no slot points; dweights [T, topk])."""
    dy, rows, weights = (np.asarray(v, dtype=np.float64) for v in (dy, rows, weights))
    live = (row_of >= 0) & (row_of < rows.shape[0])
    drows, dweights = np.zeros_like(rows), np.zeros(row_of.shape)
    for k in range(row_of.shape[1]):
        t = np.nonzero(live[:, k])[0]
        drows[row_of[t, k]] = weights[t, k, None] * dy[t]
        dweights[t, k] = (dy[t] * rows[row_of[t, k]]).sum(axis=1)
    return drows, dweights
