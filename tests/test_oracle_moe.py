"""Pins of the router's, the rows' and the 4-bit products' oracles: library results, differences, hand-worked values."""

import numpy as np
import pytest
import torch

import oracle


def test_route_by_hand():
    l = np.log(np.array([[1.0, 3.0, 3.0, 1.0], [4.0, 2.0, 1.0, 1.0]]))
    e, w = oracle.route(l, 2)
    assert e.tolist() == [[1, 2], [0, 1]]                              # equal ones: the lower first
    np.testing.assert_allclose(w, [[0.5, 0.5], [2 / 3, 1 / 3]], rtol=1e-12)
    _, w = oracle.route(l, 2, normalize=False, scale=2.0)
    np.testing.assert_allclose(w, [[0.75, 0.75], [1.0, 0.5]], rtol=1e-12)
    e, w = oracle.route(l, 2, bias=[0.0, 0.0, 0.0, 0.3], normalize=False)
    assert e.tolist() == [[3, 1], [0, 3]]
    np.testing.assert_allclose(w, [[0.125, 0.375], [0.5, 0.125]], rtol=1e-12)
    e, w = oracle.route(np.zeros((1, 2)), 1, "sigmoid", normalize=False)
    assert e.tolist() == [[0]] and w.tolist() == [[0.5]]


def test_route_masked():
    inf = np.inf
    e, w = oracle.route([[-inf, 0.0, -inf], [-inf, -inf, -inf], [np.nan, 1.0, 1.0]], 2)
    assert e.tolist() == [[1, -1], [-1, -1], [1, 2]]
    assert w[:2].tolist() == [[1.0, 0.0], [0.0, 0.0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_is_the_forward_s_differences(score, normalize):
    rng = np.random.default_rng([201, normalize, len(score)])
    l, dw = rng.standard_normal((4, 7)), rng.standard_normal((4, 3))
    l[1, 2] = -np.inf
    l[3, 1:] = -np.inf                                                 # one expert left, two slots without
    experts, _ = oracle.route(l, 3, score)
    d = oracle.route_backward(l, experts, dw, score, normalize, 1.5)
    loss = lambda x: 1.5 * (oracle.shares(oracle.scores(x, score), experts, normalize) * dw).sum()  # noqa: E731
    for i in np.ndindex(l.shape):
        if np.isinf(l[i]):
            assert d[i] == 0
            continue
        h = np.zeros_like(l)
        h[i] = 1e-5
        assert abs((loss(l + h) - loss(l - h)) / 2e-5 - d[i]) < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_matches_the_library_in_float64(score, normalize):
    rng = np.random.default_rng([202, normalize, len(score)])
    l, dw = rng.standard_normal((6, 11)) * 3, rng.standard_normal((6, 4))
    t = torch.from_numpy(l).requires_grad_(True)
    s = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    top, at = torch.topk(s, 4, dim=1)
    w = top / top.sum(1, keepdim=True) if normalize else top
    e, got = oracle.route(l, 4, score, None, normalize)
    assert np.array_equal(e, at.numpy())
    np.testing.assert_allclose(got, w.detach().numpy(), rtol=1e-12)
    w.backward(torch.from_numpy(dw))
    np.testing.assert_allclose(oracle.route_backward(l, e, dw, score, normalize), t.grad.numpy(), rtol=1e-9, atol=1e-14)


def test_sort_by_hand():
    m, row, slot = oracle.sort_slots(np.array([[2, 0], [-1, 2], [0, 5]]), 3)
    assert m.tolist() == [2, 0, 2]
    assert row.tolist() == [2, 0, -1, 3, 1, -1]
    assert slot.tolist() == [1, 4, 0, 3, -1, -1]


def test_combine_gradients_are_differences():
    rng = np.random.default_rng(203)
    row_of = np.array([[3, 0], [-1, 2], [1, 9]])                       # a slot without a row, one outside
    rows, w, dy = rng.standard_normal((4, 5)), rng.standard_normal((3, 2)), rng.standard_normal((3, 5))
    drows, dw = oracle.combine_backward(dy, rows, row_of, w)
    loss = lambda r, v: (oracle.combine(r, row_of, v) * dy).sum()      # noqa: E731
    for i in np.ndindex(rows.shape):
        h = np.zeros_like(rows)
        h[i] = 1e-6
        assert abs((loss(rows + h, w) - loss(rows - h, w)) / 2e-6 - drows[i]) < 1e-8
    for i in np.ndindex(w.shape):
        h = np.zeros_like(w)
        h[i] = 1e-6
        assert abs((loss(rows, w + h) - loss(rows, w - h)) / 2e-6 - dw[i]) < 1e-8
    assert dw[1, 0] == 0 and dw[2, 1] == 0


def test_dispatch_gradient_is_the_combine_without_weights():
    """sum over rows of dy[row] x[token of row] is sum over tokens of combine(dy)[t] x[t] for every x."""
    rng = np.random.default_rng(204)
    row_of = np.array([[3, 0], [-1, 2], [1, -1]])
    dy, x = rng.standard_normal((4, 5)), rng.standard_normal((3, 5))
    y = np.zeros((4, 5))
    for t, k in np.argwhere(row_of >= 0):
        y[row_of[t, k]] = x[t]
    assert abs((dy * y).sum() - (oracle.combine(dy, row_of) * x).sum()) < 1e-12


def test_e2m1_codes():
    assert oracle.e2m1_decode(np.arange(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert oracle.e2m1_decode(np.arange(8, 16)).tolist() == [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_w4_values_by_hand():
    w = np.array([[0x21, 0xF0]], dtype=np.uint8)                       # codes 1, 2, 0, 15
    assert oracle.unpack_codes(w).tolist() == [[1, 2, 0, 15]]
    assert oracle.w4_values(w, [[2.0, 0.5]]).tolist() == [[-14.0, -12.0, -4.0, 3.5]]
    assert oracle.w4_values(w, [[2.0, 0.5]], zero=[[1, 15]]).tolist() == [[0.0, 2.0, -7.5, 0.0]]
    assert oracle.w4_values(w, [[2.0, 0.5]], "e2m1").tolist() == [[1.0, 2.0, 0.0, -3.0]]
    p, s = oracle.w4_gemm([[1.0, -1.0, 2.0, 0.0]], w, [[2.0, 0.5]], bias=[3.0])
    assert p.tolist() == [[-14.0 + 12.0 - 8.0 + 3.0]]
    assert s.tolist() == [[2 * 9.0 + 2 * 10.0 + 0.5 * 8 * 2]]
