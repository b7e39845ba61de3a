"""GPU tests of the products with 4-bit weights against the 64-bit oracle."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
REL = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
ABS = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}
U = 2.0 ** -24


def te():
    import mxfp8_mixed_precision_amd as m
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


class Weights:
    """Random codes, scales and zero points of [rows, K] weights, on both sides."""

    def __init__(self, seed, rows, k, group, fmt="int4", scales="bf16", zeros=False):
        rng = np.random.default_rng([401, seed])
        self.fmt = fmt
        self.codes = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
        if scales == "e8m0":
            s = rng.integers(118, 126, (rows, k // group)).astype(np.uint8)
            self.values, self.s = 2.0 ** (s.astype(np.float64) - 127), torch.from_numpy(s).cuda()
        else:
            self.s = torch.from_numpy(rng.uniform(0.002, 0.02, (rows, k // group)).astype(np.float32)).cuda().to(DTYPES[scales])
            self.values = f64(self.s)
        self.z = rng.integers(0, 16, (rows, k // group), dtype=np.uint8) if zeros else None
        self.w = torch.from_numpy(self.codes).cuda()
        self.zero = None if self.z is None else torch.from_numpy(self.z).cuda()

    def rows(self, a, b):
        z = None if self.z is None else self.z[a:b]
        return self.codes[a:b], self.values[a:b], self.fmt, z


def activations(seed, m, k, dtype):
    rng = np.random.default_rng([402, seed])
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[:, rng.random(k) < 0.02] *= 20
    return torch.from_numpy(x).cuda().to(DTYPES[dtype])


def tolerance(p, s, k, group, dtype):
    """An output's rounding, and a rounding for each addition of fp32: the products of 8 weights and 8 values enter an
    accumulator together (K / 8 additions at most on a chain, with the groups' scalings, the waves' sums and the bias)."""
    return REL[dtype] * np.abs(p) + ABS[dtype] + (k / 8 + 2 * k / group + 16) * U * s


def check(got, x, w, bias, k, group, dtype, act=None, n=None):
    p, s = oracle.w4_gemm(f64(x), *w, bias)
    s = s + (0 if bias is None else np.abs(bias))
    if act is None:
        assert (np.abs(got - p) <= tolerance(p, s, k, group, dtype)).all()
        return
    # D = act(a) b: the errors of a and b through act (slope at most 1.13) and the product; act itself to 8 roundings
    e = tolerance(0 * p, s, k, group, "fp32")
    ea, eb = e[:, :n], e[:, n:]
    a, b = oracle.activation(p[:, :n], act), p[:, n:]
    d = a * b
    err = 1.13 * ea * np.abs(b) + np.abs(a) * eb + 1.13 * ea * eb + 8 * U * np.abs(d)
    assert (np.abs(got - d) <= REL[dtype] * np.abs(d) + ABS[dtype] + err * (1 + REL[dtype])).all()


SHAPES = [(1, 16, 32, 32), (1, 1, 128, 128), (3, 17, 64, 32), (16, 48, 160, 32), (17, 33, 1024, 64), (5, 100, 2080, 32),
          (31, 64, 1152, 128), (33, 40, 512, 256), (64, 129, 640, 128), (65, 20, 384, 96), (150, 16, 2048, 2048),
          (2, 200, 4096, 128)]
KINDS = [("int4", "own", False), ("int4", "fp32", True), ("int4", "own", True), ("int4", "e8m0", False),
         ("e2m1", "e8m0", False), ("e2m1", "own", False), ("e2m1", "fp32", False)]


@pytest.mark.parametrize("m,n,k,group", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_w4_gemm(m, n, k, group, dtype):
    for i, (fmt, scales, zeros) in enumerate(KINDS):
        w = Weights(i, n, k, group, fmt, dtype if scales == "own" else scales, zeros)
        x = activations(m, m, k, dtype)
        bias = activations(9, 1, n, dtype)[0] if i % 2 else None
        for out in (dtype, "fp32"):
            d = te().w4_gemm(x, w.w, fmt, w.s, w.zero, bias, out_dtype=DTYPES[out])
            assert d.dtype == DTYPES[out]
            check(f64(d), x, w.rows(0, n), None if bias is None else f64(bias), k, group, out)


@pytest.mark.parametrize("m", [1, 4])
@pytest.mark.parametrize("n,k,group", [(40, 12448, 32), (33, 10240, 128), (17, 8352, 96), (12304, 8352, 32),
                                       (24592, 8320, 64)])
def test_w4_gemm_of_a_long_k(m, n, k, group):
    """K of several chunks, with few and many tiles; the first and the last columns."""
    for i, (fmt, scales, zeros) in enumerate([("int4", "bf16", True), ("e2m1", "e8m0", False)]):
        w = Weights(20 + i, n, k, group, fmt, scales, zeros)
        x = activations(m, m, k, "bf16")
        d = te().w4_gemm(x, w.w, fmt, w.s, w.zero, out_dtype=torch.float32)
        for a, b in ((0, 24), (n - 17, n)):
            b = min(b, n)
            check(f64(d[:, a:b]), x, w.rows(a, b), None, k, group, "fp32")


@pytest.mark.parametrize("m", [1, 3, 16, 40])
@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
def test_w4_gemm_of_subnormal_activations(m, fmt):
    """fp16 below 2^-14: whole multiples of 2^-24, none of them lost."""
    w = Weights(17, 50, 416, 32, fmt, "fp32")
    rng = np.random.default_rng([403, m])
    x = torch.from_numpy((rng.integers(-1023, 1024, (m, 416)) * 2.0 ** -24).astype(np.float16)).cuda()
    assert np.abs(f64(x)).max() < 2.0 ** -14
    d = te().w4_gemm(x, w.w, fmt, w.s, out_dtype=torch.float32)
    check(f64(d), x, w.rows(0, 50), None, 416, 32, "fp32")


@pytest.mark.parametrize("m", [1, 3, 16, 40])
@pytest.mark.parametrize("fmt,scales,zeros", [("int4", "bf16", False), ("int4", "fp32", True), ("int4", "e8m0", 255),
                                              ("e2m1", "e8m0", False)])
@pytest.mark.parametrize("k,group", [(416, 32), (1024, 128), (576, 96)])
def test_w4_gemm_of_the_largest_activations(m, fmt, scales, zeros, k, group):
    """bf16 up to its largest value, where sum x q and z sum x pass fp32's range and the results do not."""
    w = Weights(18, 50, k, group, fmt, scales, bool(zeros))
    if zeros == 255:
        w.z[:] = 255
        w.zero = torch.from_numpy(w.z).cuda()
    if scales != "e8m0":                                               # 0.002 .. 0.02 over 32, so that sums stay in range
        w.s = w.s / 32
        w.values = f64(w.s)
    else:
        w.s = w.s - 20
        w.values = 2.0 ** (w.s.cpu().numpy().astype(np.float64) - 127)
    rng = np.random.default_rng([404, m])
    x = rng.choice([-1.0, 1.0], (m, k)) * rng.uniform(0.5, 1.0, (m, k)) * 3.3e38
    x = torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    d = te().w4_gemm(x, w.w, fmt, w.s, w.zero, out_dtype=torch.float32)
    assert torch.isfinite(d).all()
    check(f64(d), x, w.rows(0, 50), None, k, group, "fp32")


@pytest.mark.parametrize("m", [1, 3, 16, 40])
@pytest.mark.parametrize("fmt,zeros", [("int4", False), ("int4", True), ("e2m1", False)])
def test_w4_gemm_of_the_smallest_activations(m, fmt, zeros):
    """bf16 around 2^-118: sums are held in steps of 2^-134 (scales of 1), off by half of one for each addition of a chain
    and each group beside their relative error."""
    w = Weights(19, 50, 416, 32, fmt, "fp32", zeros)
    w.s = torch.ones_like(w.s)
    w.values = f64(w.s)
    rng = np.random.default_rng([405, m])
    x = torch.from_numpy((rng.standard_normal((m, 416)) * 2.0 ** -118).astype(np.float32)).cuda().bfloat16()
    d = te().w4_gemm(x, w.w, fmt, w.s, w.zero, out_dtype=torch.float32)
    p, s = oracle.w4_gemm(f64(x), *w.rows(0, 50), None)
    steps = 416 / 8 + 2 * 416 / 32 + 16
    most = 1 + (15 if zeros else 8 if fmt == "int4" else 0)            # the zero point multiplies its sum's error
    assert (np.abs(f64(d) - p) <= tolerance(p, s, 416, 32, "fp32") + steps * most * 2.0 ** -135).all()


@pytest.mark.parametrize("m,n,k,group", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_w4_gated_gemm(m, n, k, group, act):
    for i, (fmt, scales, zeros) in enumerate(KINDS):
        dtype = ("bf16", "fp16")[i % 2]
        w = Weights(10 + i, 2 * n, k, group, fmt, dtype if scales == "own" else scales, zeros)
        x = activations(m, m, k, dtype) * 0.25
        bias = activations(8, 1, 2 * n, dtype)[0] if i % 3 == 0 else None
        d = te().w4_gemm(x, w.w, fmt, w.s, w.zero, bias, activation=act)
        check(f64(d), x, w.rows(0, 2 * n), None if bias is None else f64(bias), k, group, dtype, act, n)


GROUPS = [([3], 16, 64, 32), ([0, 1, 0, 2], 20, 128, 64), ([5, 0, 70, 1, 16, 17], 33, 256, 128), ([0, 0], 16, 32, 32),
          ([1] * 40, 24, 160, 32), ([2, 130], 16, 512, 32)]


@pytest.mark.parametrize("splits,n,k,group", GROUPS)
@pytest.mark.parametrize("act", [None, "silu"])
def test_w4_grouped_gemm(splits, n, k, group, act):
    rows = 2 * n if act else n
    G, total = len(splits), sum(splits) + 3                            # rows behind the last group
    for i, (fmt, scales, zeros) in enumerate(KINDS[::2] + KINDS[4:5]):
        dtype = ("bf16", "fp16")[i % 2]
        w = Weights(20 + i, G * rows, k, group, fmt, dtype if scales == "own" else scales, zeros)
        x = activations(3, total, k, dtype) * 0.25
        bias = activations(7, G, rows, dtype) if i % 2 else None
        d = torch.full((total, n), 55.0, dtype=DTYPES[dtype], device="cuda")
        m = torch.tensor(splits, dtype=torch.int32, device="cuda")
        call = te().te_w4_grouped_gated_gemm if act else te().te_w4_grouped_gemm
        call(m, x, w.w, fmt, w.s, n, d, *([act] if act else []), zero=w.zero, bias=bias)
        at = 0
        for g, rows_g in enumerate(splits):
            if rows_g:
                check(f64(d)[at:at + rows_g], x[at:at + rows_g], w.rows(g * rows, (g + 1) * rows),
                      None if bias is None else f64(bias)[g], k, group, dtype, act, n)
            at += rows_g
        assert (f64(d)[at:] == 55.0).all()


def test_w4_empty_sizes():
    w = Weights(30, 16, 64, 32)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    assert te().w4_gemm(x, w.w, "int4", w.s).shape == (0, 16)
    x = torch.zeros((2, 0), dtype=torch.bfloat16, device="cuda")
    bias = torch.arange(16, dtype=torch.bfloat16, device="cuda")
    d = te().w4_gemm(x, w.w[:, :0].contiguous(), "int4", w.s[:, :0].contiguous(), None, bias)
    assert torch.equal(d, bias.expand(2, 16))


def test_w4_bad_splits_stay_inside():
    w = Weights(31, 3 * 16, 64, 32)
    big = torch.full((40, 16), 55.0, dtype=torch.bfloat16, device="cuda")
    x = activations(4, 8, 64, "bf16")
    for splits in ([100, 1, 1], [-5, 4, 100], [1 << 30, 1 << 30, 1 << 30], [2, -(1 << 31), 3]):
        te().te_w4_grouped_gemm(torch.tensor(splits, dtype=torch.int32, device="cuda"), x, w.w, "int4", w.s, 16, big[16:24])
        got = f64(big)
        assert (got[:16] == 55.0).all() and (got[24:] == 55.0).all() and np.isfinite(got).all()


def test_w4_non_finite_values_stay_in_their_rows_and_columns():
    n, k = 40, 256
    for fmt, scales in (("int4", "bf16"), ("e2m1", "e8m0")):
        w = Weights(32, n, k, 32, fmt, scales)
        x = activations(5, 20, k, "bf16")
        want = te().w4_gemm(x, w.w, fmt, w.s)
        x[3, 17], x[18, 200] = float("nan"), float("inf")
        w.s[7, 2] = 255 if scales == "e8m0" else float("nan")
        d = f64(te().w4_gemm(x, w.w, fmt, w.s))
        assert np.isnan(d[3]).all() and not np.isfinite(d[18]).any() and np.isnan(d[:, 7]).all()
        keep = np.ones((20, n), dtype=bool)
        keep[[3, 18]] = False
        keep[:, 7] = False
        assert np.array_equal(d[keep], f64(want)[keep])


def test_w4_rows_are_the_same_in_any_batch():
    """A row's result does not depend on the rows beside it, within one launch shape, nor on the call."""
    w = Weights(33, 80, 512, 128, zeros=True)
    x = activations(6, 16, 512, "bf16")
    whole = te().w4_gemm(x, w.w, "int4", w.s, w.zero)
    for m in (1, 5, 16):
        assert torch.equal(te().w4_gemm(x[:m].contiguous(), w.w, "int4", w.s, w.zero), whole[:m])
