"""The gated feed-forward GEMMs (forward, backward, grouped) on the GPU against the float64 oracle.

Tolerances.  A pre-activation P (and the backward's product) is off by at most
  eP = H + (K/16 + 12) 2^-24 (S + |bias|),   S = sum_k |a_k b_k|,
H the scaled MFMA's truncation bound (tests/mfma_model.py), K/16 its fp32 additions, and 12 for the bias, the
joining of partial sums over K and their last additions.  Then, with f the activation, its slope at most 1.13, and
2^-15 covering the fp32 evaluation (the exponential's argument, at most 150 before its result flushes to 0, is
formed with 3 roundings: 3 * 150 * ln 2 = 312 half steps of the exponential, 2^-15.7; reciprocal and products the
rest):
  aux: eP, then 2^-8 |P| for bf16
  D = f(g) u:        1.13 eg |u| + |f(g)| eu + 1.13 eg eu + 2^-15 |D|, then 2^-8 |D|
  acc u f'(g):       ea |u f'(g)| + 2^-15 |acc u| (1 + |f'|), then 2^-8 |D|      (g, u: the bf16 values given)
  acc f(g):          ea |f(g)| + 2^-15 |D|, then 2^-8 |D|
Flushing: s = 1 / (1 + e) and s (1 - s) are off by up to 2^-126 where they lie below it (the reciprocal flushes), and
f multiplies s by |g|, f' multiplies s (1 - s) by at most 2 |g| (0.8 + 0.11 g^2) < (1 + |g|)^3 (GELU; silu: |g|).  So f
is off by at most 2^-126 (1 + |g|) and f' by 2^-126 (1 + (1 + |g|)^3), and each product that follows by 2^-126 more.
"""

import numpy as np
import pytest
import torch

import mfma_model
import oracle
import workloads
from gpu_util import bf16_rne, bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu

FMTS = {"e4m3": oracle.E4M3, "e5m2": oracle.E5M2}
FLUSH = 2.0 ** -126


def te():
    import mxfp8_mixed_precision_amd as m
    return m


def operand(seed, rows, k, fmt, sigma=1.0, outliers=0.0):
    """MXFP8 codes and scales as numpy arrays."""
    x = workloads.normal_bf16(60, seed, (rows, max(k, 1)), sigma, outliers)[:, :k]
    if k == 0:
        return np.zeros((rows, 0), np.uint8), np.zeros((rows, 0), np.uint8)
    return oracle.quantize_rowwise(np.ascontiguousarray(x), FMTS[fmt])


class Forward:
    """Inputs of one forward case, its reference and its bounds."""

    def __init__(self, M, N, K, fa="e4m3", fb="e4m3", act="silu", bias=True, seed=0):
        self.M, self.N, self.K, self.fa, self.fb, self.act = M, N, K, fa, fb, act
        self.qa, self.sa = operand(seed, M, K, fa, 1.0, 0.02)
        self.qb, self.sb = operand(seed + 1, 2 * N, K, fb, 0.08)
        self.bias = workloads.normal_bf16(60, seed + 2, (2 * N,), 0.5) if bias else None
        b = bf16_to_f64(self.bias) if bias else np.zeros(2 * N)
        if K:
            self.y, _, s = oracle.mx_gemm(self.qa, self.sa, FMTS[fa], self.qb, self.sb, FMTS[fb])
            h = mfma_model.truncation_bound(self.qa, self.sa, FMTS[fa], self.qb, self.sb, FMTS[fb])
        else:
            self.y, s, h = np.zeros((M, 2 * N)), np.zeros((M, 2 * N)), 0.0
        self.p = self.y + b
        self.e = h + (K / 16 + 12) * 2.0 ** -24 * (s + np.abs(b))

    def run(self, out=None, aux=True, workspace=False):
        m = te()
        M, N = self.M, self.N
        d = torch.full((M, N), 0x55, dtype=torch.uint8 if out else torch.int16, device="cuda")
        ds = torch.full((M, N // 32), 0x55, dtype=torch.uint8, device="cuda") if out else None
        a = torch.full((M, 2 * N), 0x55, dtype=torch.int16, device="cuda") if aux else None
        ws = None
        if workspace:
            ws = torch.empty(max(m.te_mxfp8_gated_gemm_workspace_size(M, N, self.K), 1), dtype=torch.uint8,
                             device="cuda")
        m.te_mxfp8_gated_gemm(dev(self.qa), dev(self.sa), self.fa, dev(self.qb), dev(self.sb), self.fb, d, self.act,
                              d_scale=ds, d_fmt=out, bias=None if self.bias is None else dev(self.bias), aux=a,
                              workspace=ws)
        torch.cuda.synchronize()
        return d, ds, a

    def check(self, d, aux):
        g, u = np.split(self.p, 2, axis=1)
        eg, eu = np.split(self.e, 2, axis=1)
        f = oracle.activation(g, self.act)
        want = f * u
        tol = 1.13 * eg * np.abs(u) + np.abs(f) * eu + 1.13 * eg * eu + 2.0 ** -15 * np.abs(want)
        tol = tol + FLUSH * (1 + (1 + np.abs(g)) * np.abs(u))
        got = bf16_to_f64(host(d))
        assert (np.abs(got - want) <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)).all()
        if aux is not None:
            got = bf16_to_f64(host(aux))
            assert (np.abs(got - self.p) <= self.e * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(self.p)).all()


SHAPES = [(1, 16, 128), (1, 64, 1152), (2, 32, 256), (3, 48, 384), (5, 16, 640), (8, 80, 512), (15, 32, 2176),
          (16, 16, 128), (17, 48, 256), (31, 144, 128), (32, 64, 1024), (33, 16, 256), (48, 96, 640), (63, 112, 128),
          (64, 64, 256), (65, 80, 384), (100, 208, 128), (127, 64, 256), (128, 128, 128), (129, 144, 512),
          (255, 16, 128), (300, 272, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward_shapes(M, N, K):
    i = SHAPES.index((M, N, K))
    c = Forward(M, N, K, act=("silu", "gelu")[i % 2], bias=i % 3 != 0, seed=10 * i)
    d, _, aux = c.run()
    c.check(d, aux)
    again, _, _ = c.run(aux=False)
    assert torch.equal(again, d)  # the saved pre-activations do not change D


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 20, 140])
def test_forward_formats(fa, fb, act, M):
    c = Forward(M, 96, 384, fa, fb, act, seed=400)
    d, _, aux = c.run()
    c.check(d, aux)


@pytest.mark.parametrize("M,N,K", [(1, 32, 128), (1, 416, 1024), (4, 64, 256), (16, 96, 384), (40, 160, 512),
                                   (64, 32, 128), (130, 288, 256)])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
def test_forward_mx_output_equals_quantize_of_d(M, N, K, out):
    m = te()
    c = Forward(M, N, K, act="silu" if out == "e4m3" else "gelu", seed=500)
    d, _, aux = c.run()
    q, s, aux2 = c.run(out)
    want = m.mxfp8_quantize(d, out, "row")
    assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and torch.equal(aux, aux2)


@pytest.mark.parametrize("M", [1, 70, 200])
def test_forward_k_zero_is_the_bias(M):
    c = Forward(M, 48, 0, seed=600)
    d, _, aux = c.run()
    c.check(d, aux)
    assert torch.equal(aux.cpu(), dev(c.bias).cpu().expand(M, 96))


@pytest.mark.parametrize("M,N,K", [(80, 80, 640), (144, 272, 1152)])
def test_tile_pre_activations_match_the_mfma_model_bit_for_bit(M, N, K):
    """M past the few-row kernels: the K order of the additions is the model's."""
    c = Forward(M, N, K, seed=700)
    acc = mfma_model.hw_gemm_fp32(c.qa, c.sa, oracle.E4M3, c.qb, c.sb, oracle.E4M3)
    b = (c.bias.astype(np.uint32) << 16).view(np.float32)
    _, _, aux = c.run()
    assert np.array_equal(host(aux), bf16_rne((acc + b[None, :]).astype(np.float32)))


def test_forward_large_values_saturate_as_the_formula():
    """Gates far in both tails: act(g) is 0 or g, nothing is NaN."""
    M, N, K = 4, 32, 128
    for act in ("silu", "gelu"):
        c = Forward(M, N, K, act=act, seed=800)
        c.bias = bf16_rne(np.concatenate([np.where(np.arange(N) % 2, 200.0, -200.0), np.ones(N)]))
        c.p = c.y + bf16_to_f64(c.bias)
        c.e = c.e + 2.0 ** -24 * 220 * 12
        d, _, _ = c.run()
        got = bf16_to_f64(host(d))
        assert np.isfinite(got).all() and (got[:, ::2] == 0).all()
        c.check(d, None)


# ---------------------------------------------------------------- backward

class Backward:
    def __init__(self, M, N, K, fa="e5m2", fb="e4m3", act="silu", seed=0, sigma=2.0):
        self.M, self.N, self.K, self.fa, self.fb, self.act = M, N, K, fa, fb, act
        self.qa, self.sa = operand(seed, M, K, fa, 0.1, 0.02)
        self.qb, self.sb = operand(seed + 1, N, K, fb, 0.08)
        self.aux = workloads.normal_bf16(61, seed + 2, (M, 2 * N), sigma)
        if K:
            self.y, _, s = oracle.mx_gemm(self.qa, self.sa, FMTS[fa], self.qb, self.sb, FMTS[fb])
            h = mfma_model.truncation_bound(self.qa, self.sa, FMTS[fa], self.qb, self.sb, FMTS[fb])
        else:
            self.y, s, h = np.zeros((M, N)), np.zeros((M, N)), 0.0
        self.e = h + (K / 16 + 12) * 2.0 ** -24 * s

    def run(self, workspace=False):
        m = te()
        d = torch.full((self.M, 2 * self.N), 0x55, dtype=torch.int16, device="cuda")
        ws = None
        if workspace:
            ws = torch.empty(max(m.te_mxfp8_dgated_gemm_workspace_size(self.M, self.N, self.K), 1), dtype=torch.uint8,
                             device="cuda")
        m.te_mxfp8_dgated_gemm(dev(self.qa), dev(self.sa), self.fa, dev(self.qb), dev(self.sb), self.fb,
                               dev(self.aux), d, self.act, workspace=ws)
        torch.cuda.synchronize()
        return d

    def check(self, d):
        p = bf16_to_f64(self.aux).reshape(self.M, 2 * self.N)
        g, u = np.split(p, 2, axis=1)
        want = oracle.gated_grad(self.y, p, self.act)
        f, df = oracle.activation(g, self.act), oracle.activation_grad(g, self.act)
        ay = np.abs(self.y)
        tg = self.e * np.abs(u * df) + 2.0 ** -15 * ay * np.abs(u) * (1 + np.abs(df)) 
        tg = tg + FLUSH * (1 + np.abs(u) * (1 + ay * (1 + (1 + np.abs(g)) ** 3)))
        tu = self.e * np.abs(f) + 2.0 ** -15 * np.abs(self.y * f) + FLUSH * (1 + ay * (2 + np.abs(g)))
        tol = np.concatenate([tg, tu], axis=1)
        got = bf16_to_f64(host(d))
        assert (np.abs(got - want) <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)).all()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_backward_shapes(M, N, K):
    i = SHAPES.index((M, N, K))
    c = Backward(M, N, K, act=("silu", "gelu")[i % 2], seed=10 * i)
    c.check(c.run())


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_formats(fa, fb, act):
    c = Backward(70, 176, 256, fa, fb, act, seed=900)
    c.check(c.run())


def test_backward_k_zero_and_far_gates():
    c = Backward(20, 48, 0, seed=910)
    assert not bf16_to_f64(host(c.run())).any()
    c = Backward(20, 48, 128, seed=920, sigma=60.0)
    d = c.run()
    assert np.isfinite(bf16_to_f64(host(d))).all()
    c.check(d)


# ---------------------------------------------------------------- grouped

GROUPS = [[5], [0, 7, 0], [130, 1, 0, 64], [16, 16, 16, 16, 16], [0, 0, 0], [300, 3]]


@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("behind", [0, 9])
def test_grouped_forward_and_backward(counts, behind):
    """Each group equals the dense definition on its own rows; rows behind the last group stay as they were."""
    m = te()
    G, N, K, act = len(counts), 80, 256, "gelu"
    used = sum(counts)
    total = used + behind
    if total == 0:
        pytest.skip("no rows at all: nothing is launched")
    splits = torch.tensor(counts, dtype=torch.int32, device="cuda")
    d = torch.full((total, N), 0x55, dtype=torch.int16, device="cuda")
    aux = torch.full((total, 2 * N), 0x55, dtype=torch.int16, device="cuda")
    parts = [Forward(max(c, 1), N, K, act=act, seed=1000 + 3 * e) for e, c in enumerate(counts)]
    rows = [np.concatenate([getattr(f, k)[:c] for f, c in zip(parts, counts)] +
                           [np.zeros((behind, getattr(parts[0], k).shape[1]), np.uint8)]) for k in ("qa", "sa")]
    qb, sb = (np.concatenate([getattr(f, k) for f in parts]) for k in ("qb", "sb"))
    bias = np.stack([f.bias for f in parts])
    m.te_mxfp8_grouped_gated_gemm(splits, dev(rows[0]), dev(rows[1]), "e4m3", dev(qb), dev(sb), "e4m3", N, d, act,
                                  bias=dev(bias), aux=aux)
    torch.cuda.synchronize()
    off = 0
    for f, c in zip(parts, counts):
        if c:
            f.check(d[off:off + c], aux[off:off + c])
        off += c
    assert (d[used:] == 0x55).all() and (aux[used:] == 0x55).all()

    back = [Backward(max(c, 1), N, K, act=act, seed=1100 + 3 * e) for e, c in enumerate(counts)]
    rows = [np.concatenate([getattr(f, k)[:c] for f, c in zip(back, counts)] +
                           [np.zeros((behind, getattr(back[0], k).shape[1]), getattr(back[0], k).dtype)])
            for k in ("qa", "sa", "aux")]
    qb, sb = (np.concatenate([getattr(f, k) for f in back]) for k in ("qb", "sb"))
    d = torch.full((total, 2 * N), 0x55, dtype=torch.int16, device="cuda")
    m.te_mxfp8_grouped_dgated_gemm(splits, dev(rows[0]), dev(rows[1]), "e5m2", dev(qb), dev(sb), "e4m3", N,
                                   dev(rows[2]), d, act)
    torch.cuda.synchronize()
    off = 0
    for f, c in zip(back, counts):
        if c:
            f.check(d[off:off + c])
        off += c
    assert (d[used:] == 0x55).all()


# ---------------------------------------------------------------- every tile gives the same bits

def quantized(seed, rows, k, fmt="e4m3", sigma=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn((rows, k), generator=g, device="cuda") * sigma).bfloat16()
    q, s, _, _ = te().mxfp8_quantize(x, fmt, "row")
    return q, s


def run_forward(a, b, act, bias, out=None, workspace=None):
    M, N = a[0].shape[0], b[0].shape[0] // 2
    d = torch.full((M, N), 0x55, dtype=torch.uint8 if out else torch.int16, device="cuda")
    ds = torch.full((M, N // 32), 0x55, dtype=torch.uint8, device="cuda") if out else None
    aux = torch.full((M, 2 * N), 0x55, dtype=torch.int16, device="cuda")
    te().te_mxfp8_gated_gemm(*a, "e4m3", *b, "e4m3", d, act, d_scale=ds, d_fmt=out, bias=bias, aux=aux,
                             workspace=workspace)
    return [t for t in (d, ds, aux) if t is not None]


def run_backward(a, b, act, aux, workspace=None):
    d = torch.full((a[0].shape[0], 2 * b[0].shape[0]), 0x55, dtype=torch.int16, device="cuda")
    te().te_mxfp8_dgated_gemm(*a, "e4m3", *b, "e4m3", aux, d, act, workspace=workspace)
    return [d]


# (M, N, K) of grids that large tiles serve: ragged in both dimensions, an odd and an even number of K steps, one K
# step; and K % 1024 == 0 grids with one and with several tiles per workgroup
LARGE = [(1300, 4128, 384), (1300, 4128, 128), (1025, 5152, 256), (2100, 2336, 4096), (2100, 3744, 2048)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("out", [None, "e4m3", "e5m2"])
def test_forward_large_grids_equal_their_rows_alone(M, N, K, out):
    m = te()
    a, b = quantized(1, M, K), quantized(2, 2 * N, K, sigma=0.05)
    bias = torch.randn(2 * N, device="cuda").bfloat16()
    act = "silu" if out else "gelu"
    got = run_forward(a, b, act, bias, out)
    size = m.te_mxfp8_gated_gemm_workspace_size(M, N, K)
    if size:
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        again = run_forward(a, b, act, bias, out, ws)
        assert all(torch.equal(x, y) for x, y in zip(got, again))
    for r0 in (0, 448, M - 100):
        rows = [t[r0:r0 + 100].clone() for t in a]
        alone = run_forward(rows, b, act, bias, out)
        assert all(torch.equal(x, y[r0:r0 + 100]) for x, y in zip(alone, got))


def test_workspaces_serve_the_large_grids():
    m = te()
    assert m.te_mxfp8_gated_gemm_workspace_size(2100, 2336, 4096) > 0
    assert m.te_mxfp8_gated_gemm_workspace_size(2100, 3744, 2048) > 0
    assert m.te_mxfp8_gated_gemm_workspace_size(2100, 3744, 384) == 0
    assert m.te_mxfp8_dgated_gemm_workspace_size(2100, 4656, 4096) > 0


@pytest.mark.parametrize("M,N,K", [(1300, 8256, 384), (1300, 8256, 128), (2100, 4656, 4096), (2100, 7472, 2048)])
def test_backward_large_grids_equal_their_rows_alone(M, N, K):
    m = te()
    a, b = quantized(3, M, K), quantized(4, N, K, sigma=0.05)
    aux = torch.randn((M, 2 * N), device="cuda").bfloat16()
    act = "silu" if K % 1024 else "gelu"
    got, = run_backward(a, b, act, aux)
    size = m.te_mxfp8_dgated_gemm_workspace_size(M, N, K)
    if size:
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(run_backward(a, b, act, aux, ws)[0], got)
    for r0 in (0, 448, M - 100):
        alone, = run_backward([t[r0:r0 + 100].clone() for t in a], b, act, aux[r0:r0 + 100].clone())
        assert torch.equal(alone, got[r0:r0 + 100])


@pytest.mark.parametrize("counts", [[700, 0, 333, 515, 90], [2000, 1, 1]])
def test_grouped_large_grids_equal_the_dense_call(counts):
    m = te()
    G, N, K, total = len(counts), 1040, 512, sum(counts)
    a, b = quantized(5, total, K), quantized(6, G * 2 * N, K, sigma=0.05)
    bias = torch.randn((G, 2 * N), device="cuda").bfloat16()
    splits = torch.tensor(counts, dtype=torch.int32, device="cuda")
    d = torch.empty((total, N), dtype=torch.int16, device="cuda")
    aux = torch.empty((total, 2 * N), dtype=torch.int16, device="cuda")
    m.te_mxfp8_grouped_gated_gemm(splits, *a, "e4m3", *b, "e4m3", N, d, "silu", bias=bias, aux=aux)
    pre = torch.randn((total, 2 * N), device="cuda").bfloat16()
    dd = torch.empty((total, 2 * N), dtype=torch.int16, device="cuda")
    m.te_mxfp8_grouped_dgated_gemm(splits, *a, "e4m3", *[t[:G * N] for t in b], "e4m3", N, pre, dd, "silu")
    off = 0
    for e, c in enumerate(counts):
        if c >= 80:
            rows = [t[off:off + c].clone() for t in a]
            be = [t[e * 2 * N:(e + 1) * 2 * N].clone() for t in b]
            want = run_forward(rows, be, "silu", bias[e].clone())
            assert torch.equal(want[0], d[off:off + c]) and torch.equal(want[1], aux[off:off + c])
            bb = [t[e * N:(e + 1) * N].clone() for t in b]
            back, = run_backward(rows, bb, "silu", pre[off:off + c].clone())
            assert torch.equal(back, dd[off:off + c])
        off += c


# last row tiles of every kind: none, 1, 64, 127, 128, 129, 255 rows; empty experts; the weights of (10, 4176, 384) fit
# the cache that decides the order of the tiles, those of the other two do not (forward), (forward and backward)
TAILS = [256, 0, 1, 320, 127, 640, 129, 511, 0, 257]


@pytest.mark.parametrize("G,N,K", [(10, 4176, 384), (40, 1040, 4096), (70, 1040, 4096)])
@pytest.mark.parametrize("behind", [0, 130])
def test_grouped_tail_tiles_equal_the_dense_call(G, N, K, behind):
    m = te()
    counts = (TAILS * 7)[:G]
    used = sum(counts)
    a, b = quantized(7, used + behind, K), quantized(8, G * 2 * N, K, sigma=0.05)
    bias = torch.randn((G, 2 * N), device="cuda").bfloat16()
    splits = torch.tensor(counts, dtype=torch.int32, device="cuda")
    d = torch.full((used + behind, N), 0x55, dtype=torch.int16, device="cuda")
    aux, dd = (torch.full((used + behind, 2 * N), 0x55, dtype=torch.int16, device="cuda") for _ in range(2))
    m.te_mxfp8_grouped_gated_gemm(splits, *a, "e4m3", *b, "e4m3", N, d, "gelu", bias=bias, aux=aux)
    pre = torch.randn((used + behind, 2 * N), device="cuda").bfloat16()
    m.te_mxfp8_grouped_dgated_gemm(splits, *a, "e4m3", *[t[:G * N] for t in b], "e4m3", N, pre, dd, "gelu")
    off = 0
    for e, c in enumerate(counts):
        if c:
            pad = max(0, 65 - c)  # the kernel of fewer rows adds in another order
            rows = [torch.nn.functional.pad(t[off:off + c], (0, 0, 0, pad)) for t in a]
            want = run_forward(rows, [t[e * 2 * N:(e + 1) * 2 * N] for t in b], "gelu", bias[e].clone())
            assert torch.equal(want[0][:c], d[off:off + c]), e
            assert torch.equal(want[1][:c], aux[off:off + c]), e
            back, = run_backward(rows, [t[e * N:(e + 1) * N] for t in b], "gelu",
                                 torch.nn.functional.pad(pre[off:off + c], (0, 0, 0, pad)))
            assert torch.equal(back[:c], dd[off:off + c]), e
        off += c
    assert (d[used:] == 0x55).all() and (aux[used:] == 0x55).all() and (dd[used:] == 0x55).all()


@pytest.mark.parametrize("N", [80, 4176])  # the small tile and the large one
def test_grouped_splits_past_the_rows_stay_inside(N):
    m = te()
    K, total = 128, 1200
    a, b = quantized(9, total, K), quantized(10, 3 * 2 * N, K, sigma=0.05)
    pre = torch.randn((total, 2 * N), device="cuda").bfloat16()
    got = []
    for counts in ([700, 0, 500], [700, -5, 2 ** 31 - 1]):
        splits = torch.tensor(counts, dtype=torch.int32, device="cuda")
        d = torch.empty((total, N), dtype=torch.int16, device="cuda")
        dd = torch.empty((total, 2 * N), dtype=torch.int16, device="cuda")
        m.te_mxfp8_grouped_gated_gemm(splits, *a, "e4m3", *b, "e4m3", N, d, "silu")
        m.te_mxfp8_grouped_dgated_gemm(splits, *a, "e4m3", *[t[:3 * N] for t in b], "e4m3", N, pre, dd, "silu")
        got.append((d, dd))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("G,most", [(63, 5), (64, 5), (65, 5), (200, 400), (1024, 3)])
def test_grouped_many_groups_equal_the_dense_call(G, most):
    m = te()
    N, K = 16, 128
    rng = np.random.default_rng([73, G])
    counts = [int(c) for c in rng.integers(0, most + 1, G)]
    total = sum(counts)
    a, b = quantized(11, total, K), quantized(12, G * 2 * N, K, sigma=0.05)
    d = torch.empty((total, N), dtype=torch.int16, device="cuda")
    m.te_mxfp8_grouped_gated_gemm(torch.tensor(counts, dtype=torch.int32, device="cuda"), *a, "e4m3", *b, "e4m3", N, d,
                                  "silu")
    off = 0
    for e, c in enumerate(counts):
        if c and (e < 3 or 60 < e < 70 or e % 50 == 0 or e > G - 4):
            pad = max(0, 65 - c)  # the kernel of fewer rows adds in another order
            rows = [torch.nn.functional.pad(t[off:off + c], (0, 0, 0, pad)) for t in a]
            want = run_forward(rows, [t[e * 2 * N:(e + 1) * 2 * N].clone() for t in b], "silu", None)
            assert torch.equal(want[0][:c], d[off:off + c]), e
        off += c
