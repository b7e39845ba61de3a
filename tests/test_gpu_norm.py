"""te_norm_forward / te_norm_backward on the GPU against the float64 oracle.

Tolerances.  u = 2^-24 is fp32's half step, h the output type's.  Every sum of n terms is taken along
paths of at most D(n) = 64 + n / 1024 fp32 additions (per thread 8 or 32 elements of a row, or n / 1024
of a long one; then 6 steps across a wave and 16 across waves), so a sum's error is at most
D u sum|terms|.  From that, with s, mean and rstd the exact values:
  mean:  em = D u mean|s|
  rstd:  relative er = (em^2 + (D + 4) u var) / (2 (var + eps)) + 4 u
  y:     |gamma| rstd (em + u |s - mean|) + |y - beta| (er + 4 u) + u |y|, then h |y|
  dx:    c1 = mean g and c2 = mean(g xh) are off by (D + 2) u mean|g| and (D + 6) u mean|g xh|;
         dx by rstd (6 u (|g| + |c1| + |xh c2|) + dc1 + |xh| dc2) + 2 u (|dskip| + |dx|), then h |dx|
  dgamma, dbeta: paths of at most R = 100 + rows / 32 additions: (R + 6) u sum|terms|, then h |value|
fp16 outputs add half of its smallest step, 2^-25.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.float32, torch.float32)]


def te():
    import mxfp8_mixed_precision_amd as m
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def make(seed, rows, cols, dt, sigma=1.0, shift=0.0):
    rng = np.random.default_rng([71, seed])
    x = rng.standard_normal((rows, cols)) * sigma + shift
    if cols > 20:
        x[:, rng.choice(cols, cols // 20, replace=False)] *= 20.0
    return torch.from_numpy(x).to(dt).cuda()


def weights(seed, cols, wt):
    rng = np.random.default_rng([72, seed])
    return (torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).to(wt).cuda(),
            torch.from_numpy(0.3 * rng.standard_normal(cols)).to(wt).cuda())


def depth(n):
    return 64 + n / 1024


def forward(x, gamma, beta, kind, eps=1e-5, residual=None, mx=None):
    """Runs the forward with everything it can write; -> dict of tensors."""
    rows, cols = x.shape
    o = {"y": torch.empty_like(x), "rstd": torch.empty(rows, device="cuda")}
    o["mean"] = torch.empty(rows, device="cuda") if kind == "layer" else None
    o["sum"] = torch.empty_like(x) if residual is not None else None
    o["q"] = torch.empty((rows, cols), dtype=torch.uint8, device="cuda") if mx else None
    o["qs"] = torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda") if mx else None
    te().te_norm_forward(kind, x, gamma, beta, eps, y=o["y"], q=o["q"], q_scale=o["qs"], q_fmt=mx or "e4m3",
                         residual=residual, sum_out=o["sum"], mean=o["mean"], rstd=o["rstd"])
    torch.cuda.synchronize()
    return o


def check_forward(x, gamma, beta, kind, o, eps=1e-5, residual=None):
    s = f64(x)
    if residual is not None:
        want = (x.cpu().float() + residual.cpu().float()).to(x.dtype)
        assert torch.equal(o["sum"].cpu(), want)
        s = want.double().numpy()
    g = f64(gamma)
    y, mean, rstd = oracle.norm_forward(s, g, None if beta is None else f64(beta), eps, kind)
    n = s.shape[1]
    d = depth(n)
    em = d * U * np.abs(s).mean(1) if kind == "layer" else np.zeros(s.shape[0])
    var = ((s - mean[:, None]) ** 2).mean(1)
    er = (em ** 2 + (d + 4) * U * var) / (2 * (var + eps)) + 4 * U
    if kind == "layer":
        assert (np.abs(f64(o["mean"]) - mean) <= em + 2 * U * np.abs(mean)).all()
    assert (np.abs(f64(o["rstd"]) / rstd - 1) <= er).all()
    b = 0.0 if beta is None else f64(beta)
    tol = np.abs(g) * rstd[:, None] * (em[:, None] + U * np.abs(s - mean[:, None]))
    tol = tol + np.abs(y - b) * (er[:, None] + 4 * U) + U * np.abs(y)
    h = HALF[x.dtype]
    assert (np.abs(f64(o["y"]) - y) <= tol * (1 + h) + h * np.abs(y) + TINY[x.dtype]).all()


# lengths around a lane's chunk, a wave's and a workgroup's share, the 32-blocks, and past the widest register path
COLS = [1, 2, 7, 8, 9, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1000, 1024, 1031, 2048, 2050, 4096,
        4104, 5003, 8192, 8200, 16384, 16390, 32768, 33000, 70001]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward_lengths(cols, kind):
    rows = 7 if cols < 5000 else 3
    for i, (dt, wt) in enumerate(TYPES):
        x = make(cols + i, rows, cols, dt, 1.5, 0.7)
        gamma, beta = weights(cols, cols, wt)
        beta = beta if kind == "layer" and i != 1 else None
        res = make(cols + 50 + i, rows, cols, dt) if i % 2 == 0 else None
        o = forward(x, gamma, beta, kind, residual=res)
        check_forward(x, gamma, beta, kind, o, residual=res)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 15, 16, 17, 64, 257, 1025])
@pytest.mark.parametrize("cols", [24, 128, 520, 1536, 6000])
def test_forward_rows(rows, cols):
    x = make(rows * 7 + cols, rows, cols, torch.bfloat16)
    gamma, beta = weights(cols, cols, torch.bfloat16)
    check_forward(x, gamma, beta, "layer", forward(x, gamma, beta, "layer"))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (17, 96), (5, 160), (9, 1056), (33, 4128), (2, 8192),
                                       (3, 20000), (2, 40000)])
def test_forward_mx_equals_quantize_of_y(fmt, rows, cols):
    m = te()
    x = make(cols, rows, cols, torch.bfloat16, 2.0)
    x[0, :32] = 0.0
    gamma, beta = weights(cols, cols, torch.float32)
    gamma[:8] = 0.0
    o = forward(x, gamma, beta, "layer", mx=fmt)
    q, s, _, _ = m.mxfp8_quantize(o["y"], fmt, "row")
    assert torch.equal(o["q"], q) and torch.equal(o["qs"], s)
    only = torch.empty_like(q), torch.empty_like(s)
    m.te_norm_forward("layer", x, gamma, beta, 1e-5, q=only[0], q_scale=only[1], q_fmt=fmt)
    assert torch.equal(only[0], q) and torch.equal(only[1], s)


def test_forward_values_that_go_wrong():
    """Far-off means, tiny and huge values, constant rows, and rows with inf or NaN beside good ones."""
    cols = 1000
    for dt in (torch.float32, torch.bfloat16):
        x = make(5, 8, cols, dt)
        x[0] += 3000.0
        x[1] *= 1e-18
        x[2] *= 1e15
        x[3] = 2.5
        gamma, beta = weights(5, cols, dt)
        good = forward(x, gamma, beta, "layer")
        check_forward(x, gamma, beta, "layer", good)
        x[4, 17] = float("inf")
        x[6, 999] = float("nan")
        o = forward(x, gamma, beta, "layer")
        assert torch.isnan(o["y"][[4, 6]]).all()
        keep = [0, 1, 2, 3, 5, 7]
        for k in ("y", "mean", "rstd"):
            assert torch.equal(o[k][keep], good[k][keep])


def test_forward_eps_zero_on_a_constant_row():
    x = torch.full((2, 40), 3.0, device="cuda")
    x[1] = torch.arange(40.0)
    gamma, beta = weights(6, 40, torch.float32)
    o = forward(x, gamma, beta, "layer", eps=0.0)
    assert torch.isinf(o["rstd"][0]) and torch.isnan(o["y"][0]).all()  # 0 * inf, as the formula says
    check_forward(x[1:], gamma, beta, "layer", {k: None if v is None else v[1:] for k, v in o.items()}, eps=0.0)


@pytest.mark.parametrize("cols", [40, 1024, 40000])
def test_forward_sum_in_place(cols):
    x, res = make(1, 6, cols, torch.bfloat16), make(2, 6, cols, torch.bfloat16)
    gamma, beta = weights(3, cols, torch.bfloat16)
    want = forward(x, gamma, beta, "layer", residual=res)
    for target in ("x", "residual"):
        t = {"x": x.clone(), "residual": res.clone()}
        y = torch.empty_like(x)
        te().te_norm_forward("layer", t["x"], gamma, beta, 1e-5, y=y, residual=t["residual"], sum_out=t[target])
        assert torch.equal(y, want["y"]) and torch.equal(t[target], want["sum"])


# ---------------------------------------------------------------- backward

def backward(dy, x, gamma, mean, rstd, kind, dskip=None, want_dbeta=True):
    m = te()
    dx, dg = torch.empty_like(x), torch.empty_like(gamma)
    db = torch.empty_like(gamma) if kind == "layer" and want_dbeta else None
    ws = torch.full((max(m.te_norm_backward_workspace_size(*x.shape), 16),), 0xFF, dtype=torch.uint8, device="cuda")
    m.te_norm_backward(kind, dy, x, gamma, mean, rstd, dx, dg, db, dskip=dskip, workspace=ws)
    torch.cuda.synchronize()
    return dx, dg, db


def check_backward(dy, x, gamma, mean, rstd, kind, got, dskip=None):
    n, rows = x.shape[1], x.shape[0]
    d64 = None if dskip is None else f64(dskip)
    m64 = None if mean is None else f64(mean)
    wdx, wdg, wdb = oracle.norm_backward(f64(dy), f64(x), f64(gamma), m64, f64(rstd), kind, d64)
    r = f64(rstd)[:, None]
    xh = (f64(x) - m64[:, None] if kind == "layer" else f64(x)) * r
    g = f64(dy) * f64(gamma)
    c1 = np.abs(g).mean(1, keepdims=True) if kind == "layer" else 0.0
    c2 = np.abs(g * xh).mean(1, keepdims=True)
    d = depth(n)
    tol = r * (6 * U * (np.abs(g) + c1 + np.abs(xh) * c2) + (d + 2) * U * c1 + np.abs(xh) * (d + 6) * U * c2)
    tol = tol + 2 * U * (np.abs(wdx) + (0.0 if dskip is None else np.abs(d64)))
    h = HALF[x.dtype]
    assert (np.abs(f64(got[0]) - wdx) <= tol * (1 + h) + h * np.abs(wdx) + TINY[x.dtype]).all()
    hw, tw = HALF[gamma.dtype], TINY[gamma.dtype]
    paths = 106 + rows / 32
    e = paths * U * np.abs(f64(dy) * xh).sum(0)
    assert (np.abs(f64(got[1]) - wdg) <= e * (1 + hw) + hw * np.abs(wdg) + tw).all()
    if got[2] is not None:
        e = paths * U * np.abs(f64(dy)).sum(0)
        assert (np.abs(f64(got[2]) - wdb) <= e * (1 + hw) + hw * np.abs(wdb) + tw).all()


def stats(x, kind):
    mean = x.double().mean(1) if kind == "layer" else torch.zeros(x.shape[0], device="cuda", dtype=torch.float64)
    rstd = 1 / torch.sqrt((x.double() - mean[:, None]).square().mean(1) + 1e-5)
    return (mean.float() if kind == "layer" else None), rstd.float()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_lengths(cols, kind):
    rows = 37 if cols < 5000 else 5
    for i, (dt, wt) in enumerate(TYPES):
        x = make(cols + i, rows, cols, dt, 1.5, 0.5)
        dy = make(cols + 9 + i, rows, cols, dt, 0.1)
        dskip = make(cols + 19 + i, rows, cols, dt, 0.1) if i % 2 else None
        gamma, _ = weights(cols, cols, wt)
        mean, rstd = stats(x, kind)
        got = backward(dy, x, gamma, mean, rstd, kind, dskip, want_dbeta=i != 2)
        check_backward(dy, x, gamma, mean, rstd, kind, got, dskip)


@pytest.mark.parametrize("rows", [1, 2, 3, 8, 31, 32, 33, 255, 256, 257, 1000, 4099, 9001])
@pytest.mark.parametrize("cols", [16, 130, 513, 2304])
def test_backward_rows(rows, cols):
    x, dy = make(rows + cols, rows, cols, torch.bfloat16), make(rows, rows, cols, torch.bfloat16, 0.1)
    gamma, _ = weights(cols, cols, torch.float32)
    mean, rstd = stats(x, "layer")
    check_backward(dy, x, gamma, mean, rstd, "layer", backward(dy, x, gamma, mean, rstd, "layer"))


def test_backward_no_rows_gives_zero_gradients():
    x = torch.empty((0, 300), device="cuda")
    gamma = torch.ones(300, device="cuda")
    e = torch.empty(0, device="cuda")
    dx, dg, db = backward(x, x, gamma, e, e, "layer")
    assert not dg.any() and not db.any()


def test_backward_is_deterministic_and_dx_may_be_dskip():
    x, dy = make(1, 700, 1111, torch.bfloat16), make(2, 700, 1111, torch.bfloat16, 0.1)
    dskip = make(3, 700, 1111, torch.bfloat16, 0.1)
    gamma, _ = weights(1, 1111, torch.float32)
    mean, rstd = stats(x, "layer")
    first = backward(dy, x, gamma, mean, rstd, "layer", dskip)
    again = backward(dy, x, gamma, mean, rstd, "layer", dskip)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    m = te()
    ws = torch.empty(m.te_norm_backward_workspace_size(700, 1111), dtype=torch.uint8, device="cuda")
    dg = torch.empty_like(gamma)
    m.te_norm_backward("layer", dy, x, gamma, mean, rstd, dskip, dg, None, dskip=dskip, workspace=ws)
    assert torch.equal(dskip, first[0]) and torch.equal(dg, first[1])


def test_backward_a_bad_row_stays_in_its_row_and_the_columns():
    x, dy = make(1, 40, 600, torch.float32), make(2, 40, 600, torch.float32, 0.1)
    gamma, _ = weights(1, 600, torch.float32)
    mean, rstd = stats(x, "layer")
    good = backward(dy, x, gamma, mean, rstd, "layer")
    dy[11, 5] = float("nan")
    got = backward(dy, x, gamma, mean, rstd, "layer")
    assert torch.isnan(got[0][11]).all()
    keep = [r for r in range(40) if r != 11]
    assert torch.equal(got[0][keep], good[0][keep])
    cols = [c for c in range(600) if c != 5]
    assert torch.equal(got[1][cols], good[1][cols]) and torch.isnan(got[1][5]) and torch.isnan(got[2][5])


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients_against_differences_of_the_forward(kind):
    """fp32, 64 bits kept in the sums: (L(x + h v) - L(x - h v)) / 2h against <dx, v>, L = sum(y dy), along random v.
    The difference's own error: the forward's y is off by at most 1e-6 max|y| (fp32), so L by
    1e-6 sum|dy||y|, divided by h; plus the h^2 term, taken as the change between h and 2h."""
    rows, cols = 4, 96
    x, dy = make(1, rows, cols, torch.float32), make(2, rows, cols, torch.float32)
    gamma, _ = weights(4, cols, torch.float32)
    o = forward(x, gamma, None, kind)
    dx, dg, _ = backward(dy, x, gamma, o["mean"], o["rstd"], kind)
    rng = np.random.default_rng(3)
    v = torch.from_numpy(rng.standard_normal((rows, cols))).float().cuda()
    w = torch.from_numpy(rng.standard_normal(cols)).float().cuda()

    def loss(a, b):
        return float((forward(a, b, None, kind)["y"].double() * dy.double()).sum())

    noise = 1e-6 * float((o["y"].double() * dy.double()).abs().sum())
    for got, at in ((float((dx.double() * v.double()).sum()), lambda t: loss(x + t * v, gamma)),
                    (float((dg.double() * w.double()).sum()), lambda t: loss(x, gamma + t * w))):
        h = 2.0 ** -6
        d1, d2 = (at(h) - at(-h)) / (2 * h), (at(2 * h) - at(-2 * h)) / (4 * h)
        assert abs(d1 - got) <= noise / h + abs(d2 - d1) + 1e-5 * abs(got)


def test_more_rows_than_one_launch_holds():
    rows = (1 << 25) + 5  # 2^21 workgroups of 16 rows, and a second launch
    x = torch.randn((rows, 2), device="cuda")
    gamma, beta = weights(8, 2, torch.float32)
    o = forward(x, gamma, beta, "layer")
    for sl in (slice(0, 40), slice((1 << 25) - 20, rows)):
        want = forward(x[sl].clone(), gamma, beta, "layer")
        for k in ("y", "mean", "rstd"):
            assert torch.equal(o[k][sl], want[k])
    dx, dg, db = backward(x, x, gamma, o["mean"], o["rstd"], "layer")
    want = backward(x[-20:].clone(), x[-20:].clone(), gamma, o["mean"][-20:].clone(), o["rstd"][-20:].clone(), "layer")
    assert torch.equal(dx[-20:], want[0])
    # dbeta: exact to the paths' rounding (at most 100 + rows / 32 additions, here far fewer: rows / 16384 + 200)
    bound = (rows / 16384 + 200) * U * x.double().abs().sum(0)
    assert ((db.double() - x.double().sum(0)).abs() <= bound).all()


@pytest.mark.parametrize("cols", [130, 1024, 2048])
def test_backward_batches_share_the_workspace_of_the_longest(cols):
    """Shorter last batches of a program that allocated once, for its longest: same bits as with a workspace of their
    own, and nothing written behind what is asked for."""
    m = te()
    longest = 4096
    size = m.te_norm_backward_workspace_size(longest, cols)
    raw = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    gamma, _ = weights(9, cols, torch.float32)
    for rows in (longest, 2047, 1023, 511, 300, 1):
        x, dy = make(rows, rows, cols, torch.bfloat16), make(rows + 1, rows, cols, torch.bfloat16, 0.1)
        mean, rstd = stats(x, "layer")
        want = backward(dy, x, gamma, mean, rstd, "layer")
        dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
        m.te_norm_backward("layer", dy, x, gamma, mean, rstd, dx, dg, db, workspace=raw[:size])
        assert torch.equal(dx, want[0]) and torch.equal(dg, want[1]) and torch.equal(db, want[2]), rows
        assert (raw[size:] == 0xA5).all()
