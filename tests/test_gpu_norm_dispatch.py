"""te_norm_forward / te_norm_backward on the GPU at sizes that reach every kernel of their launch rules with more rows
than CUs, against the float64 oracle (tolerances: test_gpu_norm.py) and the rowwise quantize."""

import pytest
import torch

from test_gpu_norm import TYPES, backward, check_backward, check_forward, forward, make, stats, te, weights

pytestmark = pytest.mark.gpu

# more rows than CUs: a wave or 256 threads per row with 1 to 4 chunks a thread, 1024 threads with 2 and 4, and the
# row that is read again; whole chunks, whole rows of threads, and odd tails of each
BATCHES = [(260, 1000), (261, 1535), (300, 1800), (257, 2048), (259, 1601), (300, 2999), (270, 4096), (261, 4099),
           (258, 6007), (300, 7000), (257, 8192), (263, 8191), (258, 12_001), (257, 20_003), (257, 33_001)]


@pytest.mark.parametrize("rows,cols", BATCHES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward_batches(rows, cols, kind):
    i = BATCHES.index((rows, cols))
    for k, (dt, wt) in enumerate((TYPES[i % 2], TYPES[2 + i % 2], TYPES[4])):
        x = make(cols + k, rows, cols, dt, 1.5, 0.7)
        gamma, beta = weights(cols, cols, wt)
        res = make(cols + 50 + k, rows, cols, dt) if (i + k + (kind == "rms")) % 2 else None
        beta = beta if kind == "layer" and (i + k) % 3 else None
        check_forward(x, gamma, beta, kind, forward(x, gamma, beta, kind, residual=res), residual=res)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(300, 96), (290, 992), (259, 1056), (300, 1536), (257, 1568), (261, 2048),
                                       (300, 2080), (257, 4096), (263, 6144), (300, 6176), (257, 8192),
                                       (259, 12_320), (257, 32_768), (258, 32_800)])
def test_forward_mx_batches_equal_quantize_of_y(rows, cols, fmt):
    """RMS norm with a residual straight to MXFP8, as a prenorm block calls it; rows of zeros, tiny values, infinities
    and NaN among them."""
    m = te()
    x, res = make(cols, rows, cols, torch.bfloat16, 2.0), make(cols + 1, rows, cols, torch.bfloat16)
    x[3], res[3] = 0.0, 0.0
    x[5] *= 2.0 ** -70
    res[5] = 0.0
    x[7, cols // 2] = float("inf")
    x[rows - 1, cols - 1] = float("nan")
    gamma, _ = weights(cols, cols, torch.bfloat16)
    gamma[32:64] = 0.0
    o = forward(x, gamma, None, "rms", residual=res, mx=fmt)
    q, s, _, _ = m.mxfp8_quantize(o["y"], fmt, "row")
    assert torch.equal(o["q"], q) and torch.equal(o["qs"], s)
    only, total = (torch.empty_like(q), torch.empty_like(s)), torch.empty_like(x)
    m.te_norm_forward("rms", x, gamma, None, 1e-5, q=only[0], q_scale=only[1], q_fmt=fmt, residual=res, sum_out=total)
    assert torch.equal(only[0], q) and torch.equal(only[1], s)
    assert torch.equal(total.view(torch.int16), o["sum"].view(torch.int16))  # bits: there is a NaN among them


# Several rows of a workgroup in turn.  512 to 1024 threads a row, four chunks a thread, and the row that is read again
# (16-bit past 16384 columns, fp32 past 8192); then every width of 1024-thread workgroups of several rows
WALKS = [(600, 4500), (1100, 5003), (600, 6000), (600, 8191), (600, 8192), (600, 8200), (515, 16_384),
         (520, 12_001), (300, 17_001)]
SHARED = [(16_500, 100), (8300, 250), (4100, 500), (2200, 1000), (1400, 1500), (1100, 2048), (700, 2500),
          (520, 4096), (1100, 3999)]


@pytest.mark.parametrize("rows,cols", WALKS + SHARED)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_walks(rows, cols, kind):
    cases = WALKS + SHARED
    i = cases.index((rows, cols)) + (kind == "rms")
    for dt, wt in (TYPES[i % 2], TYPES[2 + i % 2], TYPES[4])[:: 1 if cols < 9000 else 2]:
        x, dy = make(cols, rows, cols, dt, 1.5, 0.5), make(cols + 9, rows, cols, dt, 0.1)
        dskip = make(cols + 19, rows, cols, dt, 0.1) if i % 2 else None
        gamma, _ = weights(cols, cols, wt)
        mean, rstd = stats(x, kind)
        got = backward(dy, x, gamma, mean, rstd, kind, dskip, want_dbeta=i % 3 != 0)
        check_backward(dy, x, gamma, mean, rstd, kind, got, dskip)
        again = backward(dy, x, gamma, mean, rstd, kind, dskip, want_dbeta=i % 3 != 0)
        assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("rows,cols", [(16_500, 100), (4100, 500), (1100, 2047), (520, 4095), (1100, 5003),
                                       (600, 8191), (520, 12_001), (300, 17_001)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_backward_walks_with_dx_in_place_of_dskip(rows, cols, dt):
    x, dy, dskip = (make(s, rows, cols, dt, 0.1) for s in (1, 2, 3))
    gamma, _ = weights(1, cols, torch.float32)
    mean, rstd = stats(x, "layer")
    want = backward(dy, x, gamma, mean, rstd, "layer", dskip)
    m = te()
    ws = torch.empty(m.te_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    dg = torch.empty_like(gamma)
    m.te_norm_backward("layer", dy, x, gamma, mean, rstd, dskip, dg, None, dskip=dskip, workspace=ws)
    assert torch.equal(dskip, want[0]) and torch.equal(dg, want[1])


@pytest.mark.parametrize("rows,cols", [(300, 2000), (300, 8000), (300, 20_000)])
def test_forward_batches_with_the_sum_in_place(rows, cols):
    x, res = make(1, rows, cols, torch.bfloat16), make(2, rows, cols, torch.bfloat16)
    gamma, beta = weights(3, cols, torch.bfloat16)
    want = forward(x, gamma, beta, "layer", residual=res)
    for target in ("x", "residual"):
        t = {"x": x.clone(), "residual": res.clone()}
        y = torch.empty_like(x)
        te().te_norm_forward("layer", t["x"], gamma, beta, 1e-5, y=y, residual=t["residual"], sum_out=t[target])
        assert torch.equal(y, want["y"]) and torch.equal(t[target], want["sum"])
