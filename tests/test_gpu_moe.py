"""GPU tests of the router, the sort of the slots and the experts' rows against the 64-bit oracle."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# a rounding: half a step, relative; half the smallest subnormal, absolute
REL = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
ABS = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}
U = 2.0 ** -24


def te():
    import mxfp8_mixed_precision_amd as m
    return m


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ router

def logits(seed, tokens, experts, dtype, masked=False):
    rng = np.random.default_rng([301, seed])
    x = rng.standard_normal((tokens, experts)) * 2
    if masked:
        x[rng.random((tokens, experts)) < 0.3] = -np.inf
        x[rng.random(tokens) < 0.2] = -np.inf
    return cuda(x, DTYPES[dtype])


def weight_tolerance(x, experts, want):
    """Of a score in fp32: the exponent's argument is off by a rounding of |l - top|, expf by 2 units in the last place
    at most, sums of up to 1024 terms by one rounding each of 16 + 6 additions in a lane and across them, and 6 more
    roundings of quotient, 1 + e, scale and output: (|l - top| + 2 2 + 22 + 6) 2^-24 relative, |l| for a sigmoid's."""
    finite = np.where(np.isfinite(x), x, 0)
    span = np.max(np.abs(finite), axis=1) + (finite.max(axis=1) - finite.min(axis=1))
    return (2 * span[:, None] + 32) * U * np.abs(want)


ROUTES = [(1, 1, 1), (1, 8, 2), (3, 32, 32 - 16), (65, 33, 4), (257, 60, 6), (64, 64, 16), (100, 128, 8), (333, 256, 8),
          (50, 257, 8), (31, 512, 17), (7, 1024, 64), (40, 100, 20), (5, 17, 17), (2049, 16, 1)]


@pytest.mark.parametrize("tokens,experts,topk", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(tokens, experts, topk, score):
    for i, (dtype, bias, normalize, masked) in enumerate([("fp32", False, True, False), ("bf16", False, False, True),
                                                           ("fp16", True, True, True), ("fp32", True, False, False),
                                                           ("bf16", True, True, False)]):
        x = logits(tokens + i, tokens, experts, dtype, masked)
        b = np.random.default_rng([302, experts]).standard_normal(experts) * 0.2 if bias else None
        b = None if b is None else b.astype(np.float32)
        got, w = te().moe_route(score, x, topk, None if b is None else cuda(b), normalize, 1.5)
        want, ww = oracle.route(f64(x), topk, score, b, normalize, 1.5)
        assert np.array_equal(host(got), want), (dtype, bias, normalize, masked)
        assert (np.abs(f64(w) - ww) <= weight_tolerance(f64(x), want, ww) + 1e-40).all(), (dtype, bias, normalize)


def low_logits(seed, experts, dtype):
    """Tokens whose logits lie far below 0, close together: sigmoids around and below the smallest float."""
    rng = np.random.default_rng([312, seed])
    base = np.array([-20.0, -80.0, -86.5, -88.5, -92.0, -104.0, -200.0, -10000.0, -65504.0, 0.5])
    x = base[:, None] + np.where(base[:, None] > -1000, rng.standard_normal((base.size, experts)) * 2, 0)
    return cuda(x, DTYPES[dtype])


def log_shares(x, experts):
    """(shares, 1 - s) of the chosen experts' sigmoids: log s = -log(1 + e^-l), and the softmax of these."""
    there = experts >= 0
    l = np.take_along_axis(x, np.where(there, experts, 0), 1)
    logs = np.where(there, -np.logaddexp(0, -l), -np.inf)
    e = np.exp(logs - logs.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True), np.exp(-np.logaddexp(0, l))


@pytest.mark.parametrize("experts,topk", [(3, 2), (40, 8), (256, 16), (300, 20)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_route_shares_of_sigmoids_below_fp32(experts, topk, dtype):
    """Shares of scores add up to the scale however small the scores are, and their gradient is the formula's.  A share: an
    exponent rounded to |l - top| 2^-24, two exponentials to 2 units in the last place, 1 + e, quotient (8 + 2 roundings of
    2^-24 and the argument's), the same of their sum with 6 additions across the lanes, the quotient and the scale."""
    x = low_logits(experts, experts, dtype)
    xs = f64(x)
    got, w = te().moe_route("sigmoid", x, topk, None, True, 2.5)
    want, _ = oracle.route(xs, topk, "softmax")                        # the scores rise with the logits
    assert np.array_equal(host(got), want)
    share, rest = log_shares(xs, want)
    top = np.take_along_axis(xs, want, 1)
    r = (2 * (top.max(1) - top.min(1)) + 2 * 12 + 8)[:, None] * U
    assert (np.abs(f64(w) - 2.5 * share) <= r * 2.5 * share).all()
    np.testing.assert_allclose(f64(w).sum(axis=1), 2.5, rtol=1e-5)
    dw = np.random.default_rng([313, experts]).standard_normal((xs.shape[0], topk)).astype(np.float32)
    g = 2.5 * dw.astype(np.float64)
    mean = (g * share).sum(axis=1, keepdims=True)
    grad, big = np.zeros_like(xs), np.zeros_like(xs)
    np.put_along_axis(grad, want, share * rest * (g - mean), 1)
    # the share's error, that of the mean (|g| times the shares') with topk additions, 1 - s to 8 roundings
    np.put_along_axis(big, want, share * rest * (np.abs(g) + (np.abs(g) * share).sum(axis=1, keepdims=True)), 1)
    d = f64(te().moe_route_backward("sigmoid", x, got, cuda(dw), True, 2.5))
    tol = REL[dtype] * np.abs(grad) + ABS[dtype] + (2 * r + (topk + 10) * U) * big
    assert (np.abs(d - grad) <= tol).all(), np.max(np.abs(d - grad) - tol)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_sigmoids_among_the_subnormals(dtype):
    """Scores below 2^-126 are whole multiples of 2^-149: off by 3 steps of the exponential, the quotient and the scale,
    beside their relative error (the exponent's argument is the logit itself; 8 roundings)."""
    x = low_logits(7, 64, dtype)
    got, w = te().moe_route("sigmoid", x, 8, None, False, 1.0)
    l = np.take_along_axis(f64(x), host(got).astype(np.int64), 1)
    s = np.exp(-np.logaddexp(0, -l))
    assert (np.abs(f64(w) - s) <= 10 * U * s + 4 * 2.0 ** -149).all()


@pytest.mark.parametrize("experts,topk", [(16, 16), (200, 9), (1024, 64)])
def test_route_equal_logits_go_to_the_lowest_expert(experts, topk):
    for value in (0.0, -3.0, 7.5):
        for bias in (None, torch.full((experts,), 0.25, device="cuda")):
            x = torch.full((5, experts), value, device="cuda")
            got, _ = te().moe_route("sigmoid", x, topk, bias)
            assert np.array_equal(host(got), np.tile(np.arange(topk), (5, 1)))
    x = torch.zeros((1, experts), device="cuda")
    x[0, ::2] = -0.0                                                   # the two zeros are one value
    got, _ = te().moe_route("softmax", x, topk)
    assert np.array_equal(host(got)[0], np.arange(topk))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_sums_that_32_bits_do_not_tell_apart(score):
    """Scores plus biases that differ by less than a float's step, in both orders."""
    rng = np.random.default_rng(303)
    x = rng.standard_normal((400, 40)).astype(np.float32)
    s = oracle.scores(x.astype(np.float64), score)
    bias = (1.0 - s[0]).astype(np.float32)                             # token 0: all sums within a rounding of 1
    x[1::2] = x[0]
    x[1::2] += rng.standard_normal((200, 40)).astype(np.float32) * np.float32(1e-7)
    got, w = te().moe_route(score, cuda(x), 10, cuda(bias), False)
    want, ww = oracle.route(x, 10, score, bias, False)
    assert np.array_equal(host(got), want)


def test_route_masked_infinite_and_nan():
    inf, nan = np.inf, np.nan
    x = np.zeros((6, 9), dtype=np.float32)
    x[0] = -inf
    x[1, 1:] = -inf
    x[2, 4] = nan
    x[3, 5] = inf
    x[4] = -200.0                                                      # far below what exp takes, but finite
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            got, w = te().moe_route(score, cuda(x), 3, None, normalize)
            got, w = host(got), f64(w)
            assert got[0].tolist() == [-1, -1, -1] and w[0].tolist() == [0, 0, 0]
            assert got[1].tolist() == [0, -1, -1] and w[1, 1:].tolist() == [0, 0]
            assert got[2].tolist() == [0, 1, 2]                        # never the NaN
            assert got[3].tolist() == [5, 0, 1]
            assert got[4].tolist() == [0, 1, 2]
            if score == "softmax":
                assert w[1, 0] == 1.0
                assert np.isnan(w[2]).all() != normalize
                np.testing.assert_allclose(w[4], 1 / 3 if normalize else 1 / 9, rtol=1e-6)
            assert got[5].tolist() == [0, 1, 2]                        # the rows beside them
            np.testing.assert_allclose(w[5], 1 / 3 if normalize else 1 / 9 if score == "softmax" else 0.5, rtol=1e-6)
    bias = np.zeros(9, dtype=np.float32)
    bias[:4] = -inf
    bias[4] = nan
    got, w = te().moe_route("softmax", cuda(x[5:]), 9, cuda(bias), True)
    assert host(got)[0].tolist() == [5, 6, 7, 8, -1, -1, -1, -1, -1]
    np.testing.assert_allclose(f64(w)[0], [0.25] * 4 + [0.0] * 5, rtol=1e-6)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("experts", [9, 300])
def test_route_slots_without_an_expert_weigh_nothing(score, normalize, experts):
    """Whatever the token's other logits are: NaN and infinite ones make the softmax NaN, but not its empty slots; with a
    bias, every sum of such a token is NaN and none of its experts is chosen."""
    x = np.full((4, experts), -np.inf, dtype=np.float32)
    x[:, 2], x[0, 5], x[1, 5], x[2, 5] = 1.0, np.nan, np.inf, -np.inf
    for dtype in ("fp32", "bf16"):
        for bias in (None, torch.zeros(experts, device="cuda")):
            e, w = te().moe_route(score, cuda(x, DTYPES[dtype]), 4, bias, normalize)
            e, w = host(e), f64(w)
            want = [[2], [5, 2], [2], [2]]
            if bias is not None and score == "softmax":
                want[:2] = [], []
            for t in range(4):
                assert e[t].tolist() == want[t] + [-1] * (4 - len(want[t]))
            assert (w[e < 0] == 0).all()
            assert np.isfinite(w[2:]).all() and (w[2:, 0] > 0).all()


def test_route_of_more_tokens_than_a_launch_takes():
    """Two launches: tokens on both sides of the border and the last ones, against the same tokens alone."""
    tokens = (1 << 25) + 1001
    g = torch.Generator(device="cuda")
    g.manual_seed(302)
    x = torch.randn((tokens, 4), generator=g, device="cuda", dtype=torch.float32).half()
    dw = torch.randn((tokens, 2), generator=g, device="cuda")
    e, w = te().moe_route("softmax", x, 2, normalize=False)
    dx = te().moe_route_backward("softmax", x, e, dw, normalize=False)
    for a in (0, (1 << 25) - 500, tokens - 64):
        part = x[a:a + 600].clone()
        pe, pw = te().moe_route("softmax", part, 2, normalize=False)
        pdx = te().moe_route_backward("softmax", part, pe, dw[a:a + 600].clone(), normalize=False)
        assert torch.equal(e[a:a + 600], pe) and torch.equal(w[a:a + 600], pw) and torch.equal(dx[a:a + 600], pdx)
    assert torch.equal(torch.gather(x, 1, e.long()), x.sort(dim=1, descending=True).values[:, :2])


def test_route_no_tokens():
    got, w = te().moe_route("softmax", torch.zeros((0, 8), device="cuda"), 2)
    assert got.shape == (0, 2) and w.shape == (0, 2)
    d = te().moe_route_backward("softmax", torch.zeros((0, 8), device="cuda"), got, w)
    assert d.shape == (0, 8)


@pytest.mark.parametrize("tokens,experts,topk", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_backward(tokens, experts, topk, score, normalize):
    for i, (dtype, masked) in enumerate([("fp32", False), ("bf16", True), ("fp16", False)]):
        x = logits(tokens + 7 * i, tokens, experts, dtype, masked)
        e, _ = te().moe_route(score, x, topk, None, normalize)
        dw = np.random.default_rng([304, tokens]).standard_normal((tokens, topk)).astype(np.float32)
        got = f64(te().moe_route_backward(score, x, e, cuda(dw), normalize, 1.5))
        want = oracle.route_backward(f64(x), host(e), dw, score, normalize, 1.5)
        # scores to weight_tolerance's relative error r; a gradient is the sum of at most topk + 1 products of |g| with
        # scores (normalize: their shares), each off by 3 r and a rounding an addition
        xs = f64(x)
        s = oracle.scores(xs, score)
        sk = oracle.shares(s, host(e), normalize)
        finite = np.where(np.isfinite(xs), xs, 0)
        r = (2 * (np.abs(finite).max(1) + finite.max(1) - finite.min(1)) + 32)[:, None] * U
        g = np.abs(dw) * 1.5
        mean = (g * sk).sum(1, keepdims=True)
        big = np.zeros_like(xs)
        for k in range(topk):
            t = np.nonzero(host(e)[:, k] >= 0)[0]
            big[t, host(e)[t, k]] += g[t, k]
        chosen = big > 0
        if normalize:
            # |dl_e| <= |w_e (g_e - mean)| (softmax), times 1 - s_e (sigmoid)
            w = np.zeros_like(xs)
            for k in range(topk):
                t = np.nonzero(host(e)[:, k] >= 0)[0]
                w[t, host(e)[t, k]] = sk[t, k]
            big = w * (big + mean) * chosen
        elif score == "softmax":
            big = s * (big + mean)
        else:
            big = s * (1 - s) * big
        # the oracle's own sums are of float64 terms: sum_j ds_j s_j, 0 in the formula with normalize, is off by a rounding
        # (2^-53) of the sum of |ds_j s_j| <= max |g| for each of topk + 4 operations, times s_e <= 1
        own = (topk + 4) * 2.0 ** -52 * g.max(axis=1, keepdims=True)
        tol = REL[dtype] * np.abs(want) + ABS[dtype] + (3 * r + (topk + 2) * U) * big + own
        assert (np.abs(got - want) <= tol).all(), (dtype, masked, np.max(np.abs(got - want) - tol))
        assert (got[~np.isfinite(xs)] == 0).all()


def test_route_backward_leaves_out_bad_slots_and_adds_equal_ones():
    x = logits(1, 3, 8, "fp32")
    e = cuda(np.array([[0, 8], [-1, 2], [5, 5]], dtype=np.int32))
    dw = cuda(np.array([[1.0, 2.0], [3.0, 4.0], [0.5, 0.25]], dtype=np.float32))
    for score in ("softmax", "sigmoid"):
        got = f64(te().moe_route_backward(score, x, e, dw, False))
        want = oracle.route_backward(f64(x), np.array([[0, -1], [-1, 2], [5, 5]]), f64(dw), score, False)
        np.testing.assert_allclose(got, want, rtol=2e-6, atol=1e-7)


# ------------------------------------------------------------------ sort

SORTS = [(0, 4), (1, 1), (1, 1024), (63, 3), (64, 2), (65, 60), (2047, 8), (2048, 32), (2049, 32), (5000, 1024),
         (16384, 256), (40000, 7), (131072, 256), (600001, 100)]


@pytest.mark.parametrize("slots,experts", SORTS)
def test_sort(slots, experts):
    rng = np.random.default_rng([305, slots])
    e = rng.integers(-1 if slots % 2 else 0, experts + slots % 2, slots).astype(np.int32)  # odd: some without a row
    e[: slots // 3] = np.sort(e[: slots // 3])
    m, row, slot = te().moe_sort(cuda(e), experts)
    for got, want in zip((m, row, slot), oracle.sort_slots(e, experts)):
        assert np.array_equal(host(got), want)


@pytest.mark.parametrize("value", [0, 5, -1, 1 << 30])
def test_sort_one_expert(value):
    e = np.full((3000, 2), value, dtype=np.int32)
    m, row, slot = te().moe_sort(cuda(e), 6)
    want = oracle.sort_slots(e, 6)
    assert np.array_equal(host(m), want[0]) and np.array_equal(host(row).reshape(-1), want[1])
    assert np.array_equal(host(slot), want[2])


def test_sort_with_a_used_workspace_and_guards():
    e = np.random.default_rng(306).integers(0, 9, 100003).astype(np.int32)
    size = te().te_moe_sort_workspace_size(e.size, 9)
    ws = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    outs = [torch.full((n + 16,), 77, dtype=torch.int32, device="cuda") for n in (9, e.size, e.size)]
    want = oracle.sort_slots(e, 9)
    x = cuda(e)
    for _ in range(2):
        te().te_moe_sort(x, *(o[:w.size] for o, w in zip(outs, want)), workspace=ws[:size])
        for o, w in zip(outs, want):
            assert np.array_equal(host(o)[:w.size], w) and (host(o)[w.size:] == 77).all()
        assert (host(ws)[size:] == 0xA5).all()


# ------------------------------------------------------------------ rows

def slots_of(seed, tokens, experts, topk, masked=False):
    rng = np.random.default_rng([307, seed])
    e = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk].astype(np.int32)
    if masked:
        e[rng.random((tokens, topk)) < 0.2] = -1
        e[rng.random(tokens) < 0.1] = -1
    _, row, slot = oracle.sort_slots(e, experts)
    return row.reshape(tokens, topk), slot


def values(seed, shape, dtype, sigma=1.0):
    rng = np.random.default_rng([308, seed])
    return cuda((rng.standard_normal(shape) * sigma).astype(np.float32), DTYPES[dtype])


ROWS = [(1, 1, 1, 1), (1, 8, 2, 4096), (3, 4, 3, 7), (5, 8, 8, 8), (17, 60, 6, 2311), (130, 16, 4, 9), (64, 8, 2, 1024),
        (33, 5, 1, 511), (9, 64, 64, 130), (300, 3, 2, 33), (2, 2, 2, 20001)]


@pytest.mark.parametrize("tokens,experts,topk,cols", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_dispatch(tokens, experts, topk, cols, dtype):
    for masked in (False, True):
        row, slot = slots_of(tokens, tokens, experts, topk, masked)
        x = values(1, (tokens, cols), dtype)
        y = torch.full((tokens * topk, cols), 99.0, dtype=DTYPES[dtype], device="cuda")
        te().te_moe_dispatch(x, cuda(row), y=y)
        want = np.full((tokens * topk, cols), 99.0)                    # rows behind the last stay
        for r, s in enumerate(slot):
            if s >= 0:
                want[r] = f64(x)[s // topk]
        assert np.array_equal(f64(y), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tokens,topk,cols", [(1, 2, 32), (7, 3, 64), (40, 8, 1024), (130, 2, 2080), (9, 4, 4096)])
def test_dispatch_to_mxfp8_is_the_quantized_rows(tokens, topk, cols, fmt):
    row, slot = slots_of(tokens, tokens, 16, topk, True)
    x = values(2, (tokens, cols), "bf16", 3.0)
    x[0, :32] = 0
    y, q, s = te().moe_dispatch(x, cuda(row), fmt)
    qx, sx, _, _ = te().mxfp8_quantize(x, fmt, "row")
    n = int((slot >= 0).sum())
    token = slot[:n] // topk
    assert np.array_equal(host(q)[:n], host(qx)[token]) and np.array_equal(host(s)[:n], host(sx)[token])
    assert np.array_equal(f64(y)[:n], f64(x)[token])
    # and the codes alone
    _, q2, s2 = te().moe_dispatch(x, cuda(row), fmt, want_y=False)
    assert np.array_equal(host(q2)[:n], host(q)[:n]) and np.array_equal(host(s2)[:n], host(s)[:n])


@pytest.mark.parametrize("tokens,experts,topk,cols", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_combine(tokens, experts, topk, cols, dtype):
    """fp32 sums of topk products: a rounding each, then the output's."""
    for masked, weighted in ((False, True), (True, True), (True, False)):
        row, _ = slots_of(tokens, tokens, experts, topk, masked)
        rows = values(3, (tokens * topk, cols), dtype)
        rows[int((row >= 0).sum()):] = float("nan")                    # rows of no slot are not read
        w = np.random.default_rng(309).standard_normal((tokens, topk)).astype(np.float32) if weighted else None
        y = te().moe_combine(rows, cuda(row), None if w is None else cuda(w))
        r = np.nan_to_num(f64(rows))
        want = oracle.combine(r, row, w)
        size = oracle.combine(np.abs(r), row, None if w is None else np.abs(w))
        tol = (REL[dtype] if dtype != "fp32" else 0) * np.abs(want) + ABS[dtype] + (topk + 1) * U * size * (1 + REL[dtype])
        assert (np.abs(f64(y) - want) <= tol).all()


@pytest.mark.parametrize("tokens,experts,topk,cols", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_combine_backward(tokens, experts, topk, cols, dtype):
    for masked in (False, True):
        row, slot = slots_of(tokens, tokens, experts, topk, masked)
        rows, dy = values(4, (tokens * topk, cols), dtype), values(5, (tokens, cols), dtype, 0.1)
        w = np.random.default_rng(310).standard_normal((tokens, topk)).astype(np.float32)
        drows = torch.full_like(rows, 99.0)
        dw = torch.empty((tokens, topk), device="cuda")
        te().te_moe_combine_backward(dy, rows, cuda(row), cuda(w), dw, drows=drows)
        _, dwant = oracle.combine_backward(f64(dy), f64(rows), row, w)
        # one product in fp32, rounded to the type: exactly
        n = int((slot >= 0).sum())
        want = (torch.from_numpy(w.reshape(-1)[slot[:n]])[:, None] * dy.cpu().float()[slot[:n] // topk]).to(DTYPES[dtype])
        assert torch.equal(drows[:n].cpu(), want)
        assert (f64(drows)[n:] == 99.0).all()
        # a dot product of cols terms: a rounding for each addition of a chain, of cols / 64 and at most 32 terms
        size = oracle.combine_backward(np.abs(f64(dy)), np.abs(f64(rows)), row, w)[1]
        assert (np.abs(f64(dw) - dwant) <= (cols / 64 + 32) * U * size + 1e-40).all()
        assert (f64(dw)[row < 0] == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tokens,topk,cols", [(1, 2, 32), (7, 3, 96), (40, 8, 1024), (130, 2, 2080), (9, 4, 4096)])
def test_combine_backward_to_mxfp8_is_the_quantized_gradient(tokens, topk, cols, fmt):
    row, slot = slots_of(tokens, tokens, 16, topk, True)
    rows, dy = values(6, (tokens * topk, cols), "bf16"), values(7, (tokens, cols), "bf16", 0.01)
    w = cuda(np.random.default_rng(311).random((tokens, topk)).astype(np.float32))
    drows, dw, q, s = te().moe_combine_backward(dy, rows, cuda(row), w, fmt)
    n = int((slot >= 0).sum())
    qd, sd, _, _ = te().mxfp8_quantize(drows[:n].contiguous(), fmt, "row")
    assert np.array_equal(host(q)[:n], host(qd)) and np.array_equal(host(s)[:n], host(sd))
    _, dw2, q2, s2 = te().moe_combine_backward(dy, rows, cuda(row), w, fmt, want_drows=False)
    assert np.array_equal(host(q2)[:n], host(q)[:n]) and np.array_equal(host(s2)[:n], host(s)[:n])
    assert torch.equal(dw2, dw)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_mxfp8_rows_of_special_values(fmt):
    """Blocks of NaN, infinities, both zeros, subnormals and the largest values: as the quantize kernel takes them."""
    x = values(10, (12, 96), "bf16")
    inf, nan, big, low = float("inf"), float("nan"), 3.3895e38, 2.0 ** -133
    for t, v in enumerate((nan, inf, -inf, 0.0, -0.0, low, -low, big, -big, 2.0 ** -126)):
        x[t, 32:64] = v
        x[t, 70] = v
    x[10], x[11, 1::2] = low, -0.0
    row, slot = slots_of(12, 12, 5, 3, False)
    ones = torch.ones((12, 3), device="cuda")
    _, q, s = te().moe_dispatch(x, cuda(row), fmt, want_y=False)
    drows, _, q2, s2 = te().moe_combine_backward(x, values(11, (36, 96), "bf16"), cuda(row), ones, fmt)
    qx, sx, _, _ = te().mxfp8_quantize(x, fmt, "row")
    token = slot // 3
    assert np.array_equal(host(q), host(qx)[token]) and np.array_equal(host(s), host(sx)[token])
    qd, sd, _, _ = te().mxfp8_quantize(drows, fmt, "row")
    assert np.array_equal(host(q2), host(qd)) and np.array_equal(host(s2), host(sd))
    same = ~np.isnan(f64(x))[token]
    assert np.array_equal(f64(drows)[same], f64(x)[token][same]) and np.isnan(f64(drows)[~same]).all()


def test_rows_outside_are_not_touched():
    """Bad row numbers are left out: nothing is read or written outside the tensors."""
    big = torch.full((40, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    y = big[16:24]
    row = cuda(np.array([[0, 8], [-2, 7], [1 << 30, -(1 << 31)]], dtype=np.int32))
    x = values(8, (3, 64), "bf16")
    te().te_moe_dispatch(x, row, y=y)
    got = f64(big)
    assert np.array_equal(got[16], f64(x)[0]) and np.array_equal(got[23], f64(x)[1])
    got[16] = got[23] = 7.0
    assert (got == 7.0).all()
    out = torch.empty((3, 64), dtype=torch.bfloat16, device="cuda")
    te().te_moe_combine(y, row, out, weights=torch.ones((3, 2), device="cuda"))
    assert np.array_equal(f64(out)[:2], f64(x)[:2]) and (f64(out)[2] == 0).all()
    dw = torch.empty((3, 2), device="cuda")
    big.fill_(7.0)
    te().te_moe_combine_backward(x, y.clone(), row, torch.ones((3, 2), device="cuda"), dw, drows=y)
    got = f64(big)
    assert np.array_equal(got[16], f64(x)[0]) and np.array_equal(got[23], f64(x)[1])
    got[16] = got[23] = 7.0
    assert (got == 7.0).all()
    assert (f64(dw)[[0, 1, 2, 2], [1, 0, 0, 1]] == 0).all()


def test_non_finite_values_stay_in_their_tokens():
    row, _ = slots_of(11, 6, 4, 2)
    rows = values(9, (12, 40), "bf16")
    rows[row[2, 1], 5] = float("nan")
    rows[row[3, 0], 6] = float("inf")
    y = f64(te().moe_combine(rows, cuda(row), torch.ones((6, 2), device="cuda")))
    bad = np.zeros((6, 40), dtype=bool)
    bad[2, 5] = bad[3, 6] = True
    assert np.isnan(y[2, 5]) and np.isinf(y[3, 6]) and np.isfinite(y[~bad]).all()
