"""The gated feed-forward GEMMs on the GPU in every kernel of their launch rules, format pair and K walk that the shapes
of test_gpu_gated.py leave out, against the float64 oracle (tolerances derived there) and the rowwise quantize."""

import numpy as np
import pytest
import torch

import mfma_model
import oracle
from gpu_util import bf16_to_f64, host
from test_gpu_gated import FLUSH, FMTS, TAILS, Backward, Forward, quantized, te

pytestmark = pytest.mark.gpu

PAIRS = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")]


# ---------------------------------------------------------------- few rows

@pytest.mark.parametrize("M", [17, 20, 32])
@pytest.mark.parametrize("N", [8192, 8208])  # 8208: the last workgroup has one of its two column groups
def test_few_rows_of_wide_layers(M, N):
    i = M + N // 16
    c = Forward(M, N, 128, *PAIRS[M % 3], act=("silu", "gelu")[i % 2], bias=M != 20, seed=2000 + i)
    d, _, aux = c.run()
    c.check(d, aux)
    again, _, _ = c.run(aux=False)
    assert torch.equal(again, d)


@pytest.mark.parametrize("M", [1, 7, 16, 17, 20, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(32, 128), (96, 640), (160, 384)])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
def test_few_rows_to_mxfp8(M, N, K, out):
    c = Forward(M, N, K, *PAIRS[M % 3], act=("silu", "gelu")[M % 2], seed=2100 + M)
    d, _, aux = c.run()
    c.check(d, aux)
    q, s, aux2 = c.run(out)
    want = te().mxfp8_quantize(d, out, "row")
    assert torch.equal(aux, aux2)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])


# a wave's second and later turns through K (8 waves: from 4096; 4 waves, more than 32 rows to MXFP8: from 2048), whole
# and ragged in the last run of 4 K steps
@pytest.mark.parametrize("M", [1, 16, 20, 33, 64])
@pytest.mark.parametrize("K", [2304, 4096, 4224, 8192, 8320, 12_416])
def test_few_rows_with_a_long_k(M, K):
    c = Forward(M, 32, K, *PAIRS[(M + K // 128) % 3], act=("silu", "gelu")[M % 2], seed=2200 + M)
    d, _, aux = c.run()
    c.check(d, aux)
    q, s, aux2 = c.run("e4m3")
    want = te().mxfp8_quantize(d, "e4m3", "row")
    if M <= 32:  # the same 8 waves: the same bits
        assert torch.equal(aux, aux2) and torch.equal(q, want[0]) and torch.equal(s, want[1])
    else:  # 4 waves add in another order
        c.check(d, aux2)
        got, f = oracle.dequantize(host(q), host(s), oracle.E4M3), bf16_to_f64(host(d))
        apart = two_runs_apart(c)
        assert (np.abs(got - f) <= apart + (np.abs(f) + apart).max(axis=1, keepdims=True) / 8).all()


def two_runs_apart(c):
    """How far two kernels' bf16 D may lie apart: each within the forward's bound of the exact one, and rounded.  (A code
    is then off by at most 1/8 of its 32-block's largest value: half a step is 2^-4 of a value, and the power-of-two
    scale that leaves the largest in 256 .. 512 cuts what lies past 448.)"""
    g, u = np.split(c.p, 2, axis=1)
    eg, eu = np.split(c.e, 2, axis=1)
    f = oracle.activation(g, c.act)
    tol = 1.13 * eg * np.abs(u) + np.abs(f) * eu + 1.13 * eg * eu + 2.0 ** -15 * np.abs(f * u)
    tol = tol + FLUSH * (1 + (1 + np.abs(g)) * np.abs(u))
    return 2 * (tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(f * u))


# ---------------------------------------------------------------- large tiles, every format pair, against the oracle

class Sample:
    """Rows and columns of a large product: the operands' parts on the host, the exact product and its bound."""

    def __init__(self, a, fa, b_rows, fb, rows, k):
        qa, sa = (host(t[rows]) for t in a)
        qb, sb = b_rows
        self.y, _, s = oracle.mx_gemm(qa, sa, FMTS[fa], qb, sb, FMTS[fb])
        self.e = mfma_model.truncation_bound(qa, sa, FMTS[fa], qb, sb, FMTS[fb])
        self.s = s
        self.k = k

    def bound(self, bias):
        return self.e + (self.k / 16 + 12) * 2.0 ** -24 * (self.s + np.abs(bias))


def spots(n, seed, count=24):
    """First, last and scattered indices below n."""
    rng = np.random.default_rng([74, seed])
    return torch.from_numpy(np.unique(np.concatenate([np.arange(2), n - 1 - np.arange(2), rng.integers(0, n, count)])))


def check_forward_spots(d, aux, a, fa, b, fb, bias, act, rows, cols, N, K, base=0):
    """base: first row of the expert's weights in b."""
    c = Forward.__new__(Forward)
    c.act = act
    at = torch.cat([base + cols, base + N + cols])
    part = Sample(a, fa, [host(t[at.cuda()]) for t in b], fb, rows.cuda(), K)
    bias64 = bf16_to_f64(host(bias))[torch.cat([cols, N + cols]).numpy()] if bias is not None else 0.0
    c.p, c.e = part.y + bias64, part.bound(bias64)
    r = rows.cuda()
    c.check(d[r][:, cols.cuda()], aux[r][:, torch.cat([cols, N + cols]).cuda()])


def check_backward_spots(d, aux, a, fa, b, fb, act, rows, cols, N, K, base=0):
    c = Backward.__new__(Backward)
    part = Sample(a, fa, [host(t[(base + cols).cuda()]) for t in b], fb, rows.cuda(), K)
    both = torch.cat([cols, N + cols]).cuda()
    c.M, c.N, c.act, c.y, c.e = len(rows), len(cols), act, part.y, part.bound(0.0)
    r = rows.cuda()
    c.aux = host(aux[r][:, both].contiguous())
    c.check(d[r][:, both])


def filled(shape, byte=0x55):
    return torch.full(shape, byte, dtype=torch.int16, device="cuda")


# 8-wave tiles (one, three and a ragged number of K steps), the small tile with 4 stages, the 4-wave tile
@pytest.mark.parametrize("M,N,K", [(1300, 4128, 128), (1300, 4128, 384), (400, 1056, 2304), (2100, 2336, 4096)])
@pytest.mark.parametrize("fa,fb", PAIRS)
def test_large_forward_formats(M, N, K, fa, fb):
    m = te()
    a, b = quantized(21, M, K, fa), quantized(22, 2 * N, K, fb, 0.05)
    bias = torch.randn(2 * N, device="cuda").bfloat16()
    act = "gelu" if fb == "e5m2" else "silu"
    size = m.te_mxfp8_gated_gemm_workspace_size(M, N, K)
    first = None
    for ws in [None] + ([torch.empty(size, dtype=torch.uint8, device="cuda")] if size else []):
        d, aux = filled((M, N)), filled((M, 2 * N))
        m.te_mxfp8_gated_gemm(*a, fa, *b, fb, d, act, bias=bias, aux=aux, workspace=ws)
        rows, cols = spots(M, K, 8), spots(N, K + 1)
        check_forward_spots(d, aux, a, fa, b, fb, bias, act, rows, cols, N, K)
        for out in ("e4m3", "e5m2"):
            q, s = (torch.empty((M, n), dtype=torch.uint8, device="cuda") for n in (N, N // 32))
            m.te_mxfp8_gated_gemm(*a, fa, *b, fb, q, act, d_scale=s, d_fmt=out, bias=bias, workspace=ws)
            want = m.mxfp8_quantize(d, out, "row")
            assert torch.equal(q, want[0]) and torch.equal(s, want[1])
        assert first is None or (torch.equal(first[0], d) and torch.equal(first[1], aux))
        first = (d, aux)


@pytest.mark.parametrize("M,N,K", [(1300, 8256, 128), (1300, 8256, 384), (400, 2080, 2304), (2100, 4656, 4096)])
@pytest.mark.parametrize("fa,fb", PAIRS)
def test_large_backward_formats(M, N, K, fa, fb):
    m = te()
    a, b = quantized(23, M, K, fa, 0.1), quantized(24, N, K, fb, 0.05)
    pre = torch.randn((M, 2 * N), device="cuda").bfloat16()
    act = "silu" if fb == "e5m2" else "gelu"
    size = m.te_mxfp8_dgated_gemm_workspace_size(M, N, K)
    first = None
    for ws in [None] + ([torch.empty(size, dtype=torch.uint8, device="cuda")] if size else []):
        d = filled((M, 2 * N))
        m.te_mxfp8_dgated_gemm(*a, fa, *b, fb, pre, d, act, workspace=ws)
        check_backward_spots(d, pre, a, fa, b, fb, act, spots(M, K, 8), spots(N, K + 1), N, K)
        assert first is None or torch.equal(first, d)
        first = d


@pytest.mark.parametrize("G,N,K", [(10, 4176, 384), (40, 1040, 4096)])  # tail tiles last, and beside their experts
@pytest.mark.parametrize("fa,fb", PAIRS)
def test_grouped_formats(G, N, K, fa, fb):
    m = te()
    counts = (TAILS * 7)[:G]
    total = sum(counts)
    a = quantized(25, total, K, fa)
    b = quantized(26, G * 2 * N, K, fb, 0.05)
    bias = torch.randn((G, 2 * N), device="cuda").bfloat16()
    splits = torch.tensor(counts, dtype=torch.int32, device="cuda")
    d, aux, dd = filled((total, N)), filled((total, 2 * N)), filled((total, 2 * N))
    m.te_mxfp8_grouped_gated_gemm(splits, *a, fa, *b, fb, N, d, "silu", bias=bias, aux=aux)
    pre = torch.randn((total, 2 * N), device="cuda").bfloat16()
    half = [t[:G * N] for t in b]
    m.te_mxfp8_grouped_dgated_gemm(splits, *a, fa, *half, fb, N, pre, dd, "silu")
    off = 0
    for e, c in enumerate(counts):
        if c and e < 10:
            rows, cols = off + torch.unique(torch.tensor([0, c // 2, c - 1])), spots(N, e, 8)
            check_forward_spots(d, aux, a, fa, b, fb, bias[e], "silu", rows, cols, N, K, base=e * 2 * N)
            check_backward_spots(dd, pre, a, fa, half, fb, "silu", rows, cols, N, K, base=e * N)
        off += c


@pytest.mark.parametrize("M,N,K", [(1, 2048, 4096), (48, 512, 2048), (300, 1040, 512), (1300, 4128, 384),
                                   (2100, 2336, 4096)])
def test_the_same_call_gives_the_same_bits(M, N, K):
    m = te()
    a, b = quantized(27, M, K), quantized(28, 2 * N, K, sigma=0.05)
    half = [t[:N] for t in b]
    splits = torch.tensor([M - M // 3, 0, M // 3], dtype=torch.int32, device="cuda")
    b3 = [t.repeat(3, 1) for t in b]
    h3 = [t[:3 * N] for t in b3]
    first = None
    for _ in range(4):
        d, _, aux = m.mxfp8_gated_gemm(*a, "e4m3", *b, "e4m3", want_aux=True)
        out = [d, aux, m.mxfp8_dgated_gemm(*a, "e4m3", *half, "e4m3", aux)]
        g, ga, gd = torch.empty_like(d), torch.empty_like(aux), torch.empty_like(aux)
        m.te_mxfp8_grouped_gated_gemm(splits, *a, "e4m3", *b3, "e4m3", N, g, aux=ga)
        m.te_mxfp8_grouped_dgated_gemm(splits, *a, "e4m3", *h3, "e4m3", N, aux, gd)
        out += [g, ga, gd]
        assert first is None or all(torch.equal(x, y) for x, y in zip(first, out))
        first = out


# ---------------------------------------------------------------- NaN operands

NAN_CODE = 0x7F  # E4M3


def nan_at(t):
    return torch.isnan(t.view(torch.bfloat16))


# few rows (8 and 4 waves, a run that ends ragged), the small tiles, the 8-wave tile, the 4-wave tile
@pytest.mark.parametrize("M,N,K", [(1, 32, 128), (7, 64, 640), (20, 8224, 128), (50, 96, 4224), (70, 96, 384),
                                   (400, 1056, 2304), (1300, 4128, 384), (2100, 2336, 4096)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_nan_operands_stay_in_their_rows_and_columns(M, N, K, act):
    m = te()
    a, b = quantized(31, M, K), quantized(32, 2 * N, K, sigma=0.05)
    size = m.te_mxfp8_gated_gemm_workspace_size(M, N, K)
    r, gate, up = M - 1, 5, N - 2

    def run(qa, qb):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        d, aux = filled((M, N)), filled((M, 2 * N))
        q, s = (torch.empty((M, n), dtype=torch.uint8, device="cuda") for n in (N, N // 32))
        m.te_mxfp8_gated_gemm(qa, a[1], "e4m3", qb, b[1], "e4m3", d, act, aux=aux, workspace=ws)
        m.te_mxfp8_gated_gemm(qa, a[1], "e4m3", qb, b[1], "e4m3", q, act, d_scale=s, d_fmt="e4m3", workspace=ws)
        want = m.mxfp8_quantize(d, "e4m3", "row")
        if not 32 < M <= 64:  # (the 4-wave few-row form adds in another order)
            assert torch.equal(q, want[0]) and torch.equal(s, want[1])
        pre = torch.ones((M, 2 * N), dtype=torch.bfloat16, device="cuda")
        dd = filled((M, 2 * N))
        m.te_mxfp8_dgated_gemm(qa, a[1], "e4m3", qb[:N], b[1][:N], "e4m3", pre, dd, act)
        return d, aux, dd

    clean = run(a[0], b[0])
    qa, qb = a[0].clone(), b[0].clone()
    qa[r, K - 3] = NAN_CODE
    qb[gate, 2] = qb[N + up, K - 1] = NAN_CODE
    got = run(qa, qb)
    bad = [torch.zeros(t.shape, dtype=torch.bool, device="cuda") for t in got]
    for t in bad:
        t[r] = True
    bad[0][:, [gate, up]] = True
    bad[1][:, [gate, N + up]] = True
    bad[2][:, [gate, N + gate]] = True
    for t, c, where in zip(got, clean, bad):
        assert torch.equal(nan_at(t), where)
        assert torch.equal(t[~where], c[~where])


def test_nan_operands_stay_in_their_groups():
    m = te()
    counts, N, K = [130, 0, 1, 300, 70], 1040, 384
    total, G = sum(counts), len(counts)
    a, b = quantized(33, total, K), quantized(34, G * 2 * N, K, sigma=0.05)
    splits = torch.tensor(counts, dtype=torch.int32, device="cuda")
    pre = torch.ones((total, 2 * N), dtype=torch.bfloat16, device="cuda")

    def run(qa, qb):
        d, aux, dd = filled((total, N)), filled((total, 2 * N)), filled((total, 2 * N))
        m.te_mxfp8_grouped_gated_gemm(splits, qa, a[1], "e4m3", qb, b[1], "e4m3", N, d, aux=aux)
        m.te_mxfp8_grouped_dgated_gemm(splits, qa, a[1], "e4m3", qb[:G * N], b[1][:G * N], "e4m3", N, pre, dd)
        return d, aux, dd

    clean = run(a[0], b[0])
    qa, qb = a[0].clone(), b[0].clone()
    qa[130] = NAN_CODE                    # group 2's only row
    qb[2 * N:4 * N] = NAN_CODE            # the weights of group 1, which has no rows (backward: those of 2 and 3)
    qb[3 * 2 * N + 7] = NAN_CODE          # forward: column 7 of group 3's gate
    got = run(qa, qb)
    bad = [torch.zeros(t.shape, dtype=torch.bool, device="cuda") for t in got]
    for t in bad:
        t[130] = True
    bad[0][131:431, 7] = bad[1][131:431, 7] = True
    bad[2][130:431] = True
    for t, c, where in zip(got, clean, bad):
        assert torch.equal(nan_at(t), where)
        assert torch.equal(t[~where], c[~where])
