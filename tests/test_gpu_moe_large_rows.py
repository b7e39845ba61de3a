"""The experts' rows where they are more than 96 MB and pass the caches: odd columns and tails in every type, rows shorter
than a chunk, 16 lanes a slot, the MXFP8 outputs; slots without a row, rows that stay as they were."""

import pytest
import torch

from test_gpu_moe import ABS, DTYPES, REL, U, te

pytestmark = pytest.mark.gpu

MB = 1 << 20
# tokens, slots, columns: a tail after whole chunks, rows at odd addresses; less than a chunk; 16 lanes a slot
ROWS = [(6000, 4, 2311), (1_300_000, 8, 5), (56_000, 4, 251)]


class Slots:
    """Tokens with a random place for each slot, some without one; rows behind the last are of no slot."""

    def __init__(self, tokens, topk, seed=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = tokens * topk
        there = torch.rand(n, generator=g, device="cuda") < 0.9
        there[:topk] = False                                           # a token without any
        order = torch.rand(n, generator=g, device="cuda").argsort()    # the slots in the order of their rows
        order = order[there[order]]
        self.rows = order.numel()
        row = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        row[order] = torch.arange(self.rows, dtype=torch.int32, device="cuda")
        self.row_of, self.slot_of, self.token_of = row.view(tokens, topk), order, order // topk
        self.total, self.g = n, g

    def randn(self, *shape, dtype="fp32", sigma=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * sigma).to(DTYPES[dtype])


def slots(tokens, topk, cols, dtype):
    size = {"fp32": 4, "bf16": 2, "fp16": 2}[dtype]
    tokens = tokens // 2 if dtype == "fp32" else tokens
    s = Slots(tokens, topk)
    assert s.total * cols * size > 96 * MB
    return s, tokens


@pytest.mark.parametrize("tokens,topk,cols", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_dispatch(tokens, topk, cols, dtype):
    s, tokens = slots(tokens, topk, cols, dtype)
    x = s.randn(tokens, cols, dtype=dtype)
    big = torch.full((s.total * cols + 64,), 99.0, dtype=DTYPES[dtype], device="cuda")
    y = big[:s.total * cols].view(s.total, cols)
    te().te_moe_dispatch(x, s.row_of, y=y)
    assert torch.equal(y[:s.rows], x[s.token_of])
    assert (big[s.rows * cols:] == 99.0).all()                         # rows of no slot, and behind the tensor


@pytest.mark.parametrize("tokens,topk,cols", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_combine(tokens, topk, cols, dtype):
    """fp32 sums of topk products: a rounding each, then the output's."""
    s, tokens = slots(tokens, topk, cols, dtype)
    rows = s.randn(s.total, cols, dtype=dtype)
    rows[s.rows:] = float("nan")                                       # rows of no slot are not read
    for w in (s.randn(tokens, topk), None):
        y = te().moe_combine(rows, s.row_of, w)
        want = torch.zeros((tokens, cols), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for k in range(topk):
            at = s.row_of[:, k].long()
            v = torch.where((at >= 0)[:, None], rows[at.clamp(min=0)].double(), 0.0)
            v = v if w is None else v * w[:, k, None].double()
            want += v
            size += v.abs()
        rel = REL[dtype] if dtype != "fp32" else 0
        tol = rel * want.abs() + ABS[dtype] + (topk + 1) * U * size * (1 + REL[dtype])
        assert bool(((y.double() - want).abs() <= tol).all())
        assert bool((y[0] == 0).all())


@pytest.mark.parametrize("tokens,topk,cols", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_combine_backward(tokens, topk, cols, dtype):
    s, tokens = slots(tokens, topk, cols, dtype)
    rows, dy = s.randn(s.total, cols, dtype=dtype), s.randn(tokens, cols, dtype=dtype, sigma=0.1)
    w = s.randn(tokens, topk)
    big = torch.full((s.total * cols + 64,), 99.0, dtype=DTYPES[dtype], device="cuda")
    drows, dw = big[:s.total * cols].view(s.total, cols), torch.empty((tokens, topk), device="cuda")
    te().te_moe_combine_backward(dy, rows, s.row_of, w, dw, drows=drows)
    # one product in fp32, rounded to the type: exactly
    want = (w.view(-1)[s.slot_of][:, None] * dy[s.token_of].float()).to(DTYPES[dtype])
    assert torch.equal(drows[:s.rows], want)
    assert (big[s.rows * cols:] == 99.0).all()
    # a dot product of cols terms: a rounding for each addition of a chain, of cols / 16 (16 lanes) and at most 32 terms
    dwant, size = torch.zeros_like(dw, dtype=torch.float64), torch.zeros_like(dw, dtype=torch.float64)
    for k in range(topk):
        at = s.row_of[:, k].long()
        v = torch.where((at >= 0)[:, None], rows[at.clamp(min=0)].double(), 0.0) * dy.double()
        dwant[:, k], size[:, k] = v.sum(1), v.abs().sum(1)
    assert bool(((dw.double() - dwant).abs() <= (cols / 16 + 32) * U * size + 1e-40).all())
    assert (dw[s.row_of < 0] == 0).all()
    # in place
    dw2 = torch.empty_like(dw)
    te().te_moe_combine_backward(dy, rows, s.row_of, w, dw2, drows=rows)
    assert torch.equal(rows[:s.rows], want) and torch.equal(dw2, dw)


@pytest.mark.parametrize("tokens,topk,cols", [(6000, 4, 2336), (60_000, 4, 224), (220_000, 8, 32)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_mxfp8_rows_are_the_quantized_ones(tokens, topk, cols, fmt):
    s, tokens = slots(tokens, topk, cols, "bf16")
    x, rows = s.randn(tokens, cols, dtype="bf16", sigma=3.0), s.randn(s.total, cols, dtype="bf16")
    x[1, :32] = 0
    w = torch.rand((tokens, topk), generator=s.g, device="cuda")

    def outputs():
        big = torch.full((s.total * cols + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        return big, big[:s.total * cols].view(s.total, cols), torch.full((s.total, cols // 32), 0x5A, dtype=torch.uint8,
                                                                         device="cuda")

    qx, sx, _, _ = te().mxfp8_quantize(x, fmt, "row")
    for want_y in (False, True):
        big, q, scale = outputs()
        y = torch.empty((s.total, cols), dtype=torch.bfloat16, device="cuda") if want_y else None
        te().te_moe_dispatch(x, s.row_of, y=y, q=q, q_scale=scale, q_fmt=fmt)
        assert torch.equal(q[:s.rows], qx[s.token_of]) and torch.equal(scale[:s.rows], sx[s.token_of])
        assert (big[s.rows * cols:] == 0x5A).all() and (scale[s.rows:] == 0x5A).all()
        assert y is None or torch.equal(y[:s.rows], x[s.token_of])
    dw = torch.empty((tokens, topk), device="cuda")
    d = (w.view(-1)[s.slot_of][:, None] * x[s.token_of].float()).bfloat16()
    qd, sd, _, _ = te().mxfp8_quantize(d, fmt, "row")
    for want_d in (False, True):
        big, q, scale = outputs()
        drows = torch.empty((s.total, cols), dtype=torch.bfloat16, device="cuda") if want_d else None
        te().te_moe_combine_backward(x, rows, s.row_of, w, dw, drows=drows, q=q, q_scale=scale, q_fmt=fmt)
        assert torch.equal(q[:s.rows], qd) and torch.equal(scale[:s.rows], sd)
        assert (big[s.rows * cols:] == 0x5A).all() and (scale[s.rows:] == 0x5A).all()
        assert drows is None or torch.equal(drows[:s.rows], d)


def test_captured_and_replayed():
    s, tokens = slots(6000, 4, 2311, "fp16")
    x, dy = s.randn(tokens, 2311, dtype="fp16"), s.randn(tokens, 2311, dtype="fp16", sigma=0.1)
    w = s.randn(tokens, 4)

    def step():
        y, _, _ = te().moe_dispatch(x, s.row_of)
        out = te().moe_combine(y, s.row_of, w)
        drows, dw, _, _ = te().moe_combine_backward(dy, y, s.row_of, w)
        return y[:s.rows], out, drows[:s.rows], dw

    want = [v.clone() for v in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for v in got:
            v.zero_()
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, eager, want):
            assert torch.equal(a, c) and torch.equal(b, c)
