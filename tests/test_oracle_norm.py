"""Pins of the norm and gated oracles: library results, invariants and differences."""

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("cols", [1, 2, 7, 64])
def test_layer_norm_matches_the_library_in_float64(cols):
    rng = np.random.default_rng([91, cols])
    x = rng.standard_normal((5, cols)) * 3 + 2
    g, b = rng.standard_normal(cols), rng.standard_normal(cols)
    y, mean, rstd = oracle.norm_forward(x, g, b, 1e-5)
    t = [torch.from_numpy(v).requires_grad_(True) for v in (x, g, b)]
    want = torch.nn.functional.layer_norm(t[0], (cols,), t[1], t[2], 1e-5)
    np.testing.assert_allclose(y, want.detach().numpy(), rtol=1e-12, atol=1e-12)
    dy = rng.standard_normal(y.shape)
    want.backward(torch.from_numpy(dy))
    got = oracle.norm_backward(dy, x, g, mean, rstd)
    for a, v in zip(got, t):
        np.testing.assert_allclose(a, v.grad.numpy(), rtol=1e-9, atol=1e-9)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_is_the_forward_s_differences(kind):
    rng = np.random.default_rng([92, len(kind)])
    x, dy = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))
    g = rng.standard_normal(6)
    _, mean, rstd = oracle.norm_forward(x, g, None, 1e-5, kind)
    dx, dg, _ = oracle.norm_backward(dy, x, g, mean, rstd, kind)
    h = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        up = (oracle.norm_forward(x + e, g, None, 1e-5, kind)[0] * dy).sum()
        dn = (oracle.norm_forward(x - e, g, None, 1e-5, kind)[0] * dy).sum()
        assert abs((up - dn) / (2 * h) - dx[i]) < 1e-7 * (1 + abs(dx[i]))
    for c in range(6):
        e = np.zeros(6)
        e[c] = h
        up = (oracle.norm_forward(x, g + e, None, 1e-5, kind)[0] * dy).sum()
        dn = (oracle.norm_forward(x, g - e, None, 1e-5, kind)[0] * dy).sum()
        assert abs((up - dn) / (2 * h) - dg[c]) < 1e-7 * (1 + abs(dg[c]))


def test_rms_norm_rows_have_unit_mean_square():
    x = np.random.default_rng(93).standard_normal((4, 50)) * 7
    y, mean, _ = oracle.norm_forward(x, np.ones(50), None, 0.0, "rms")
    np.testing.assert_allclose((y * y).mean(axis=1), 1.0, rtol=1e-12)
    assert not mean.any()


def test_activations_match_the_library_in_float64():
    x = np.linspace(-30, 30, 1201)
    t = torch.from_numpy(x).requires_grad_(True)
    for act, fn in (("silu", torch.nn.functional.silu),
                    ("gelu", lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        want = fn(t)
        t.grad = None
        want.sum().backward()
        np.testing.assert_allclose(oracle.activation(x, act), want.detach().numpy(), rtol=1e-9, atol=1e-14)
        np.testing.assert_allclose(oracle.activation_grad(x, act), t.grad.numpy(), rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_is_the_forward_s_differences(act):
    rng = np.random.default_rng(94)
    p, dh = rng.standard_normal((2, 8)), rng.standard_normal((2, 4))
    got = oracle.gated_grad(dh, p, act)
    h = 1e-6
    for i in np.ndindex(p.shape):
        e = np.zeros_like(p)
        e[i] = h
        diff = ((oracle.gated(p + e, act) - oracle.gated(p - e, act)) * dh).sum() / (2 * h)
        assert abs(diff - got[i]) < 1e-8 * (1 + abs(got[i]))
