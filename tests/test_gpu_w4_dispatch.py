"""The GEMMs with 4-bit weights in every kernel of their launch rules, and in walks of K of more than one span, that the
shapes of test_gpu_w4.py leave out (256 CUs), against the float64 oracle within the bound derived there."""

import numpy as np
import pytest
import torch

from test_gpu_w4 import DTYPES, Weights, activations, check, f64, te

pytestmark = pytest.mark.gpu

# code format, activations and bias, scales, zero points
KINDS = [("int4", "bf16", "bf16", True), ("e2m1", "bf16", "e8m0", False), ("int4", "fp16", "fp32", False),
         ("e2m1", "fp16", "fp16", False)]


def rows_of(w, i):
    return w.codes[i], w.values[i], w.fmt, None if w.z is None else w.z[i]


def run(seed, m, n, k, group, kind, act=None, bias=False):
    """The first and the last columns against the oracle, all of them finite."""
    fmt, dtype, scales, zeros = kind
    rows = 2 * n if act else n
    w = Weights(seed, rows, k, group, fmt, scales, zeros)
    x = activations(m, m, k, dtype) * 0.25
    b = activations(9, 1, rows, dtype)[0] if bias else None
    d = te().w4_gemm(x, w.w, fmt, w.s, w.zero, b, act)
    assert d.dtype == DTYPES[dtype] and torch.isfinite(d).all()
    for a, e in ((0, min(24, n)), (max(0, n - 19), n)):
        i = np.concatenate([np.arange(a, e), n + np.arange(a, e)]) if act else np.arange(a, e)
        check(f64(d[:, a:e]), x, rows_of(w, i), None if b is None else f64(b)[i], k, group, dtype, act, e - a)
    return d


# ---------------------------------------------------------------- many tiles of columns

# 769 tiles of 16 columns: plain 12291, gated 12291; plain 24600 in tiles of 32.  K: one step and less, one chunk and a
# tail, two chunks (of 32 steps, of 64 from K = 6144 on; two to four rows and K up to 2048: one of 16); groups of a block,
# of steps, of others
@pytest.mark.parametrize("n,act", [(12_291, None), (12_291, "silu"), (24_600, None)])
@pytest.mark.parametrize("m,k,group", [(1, 96, 32), (1, 416, 32), (1, 2112, 96), (1, 5248, 128), (1, 5152, 32),
                                       (1, 6240, 96), (1, 6272, 128),
                                       (3, 96, 96), (4, 1056, 32), (2, 2016, 96), (3, 2048, 128), (4, 2080, 32)])
def test_few_rows_of_wide_layers(m, n, k, group, act):
    for kind in KINDS:
        run(m + k, m, n, k, group, kind, act, bias=m % 2 == 1)


# 385 tiles of columns with one of rows, and 129 with three
@pytest.mark.parametrize("n,act", [(6160, None), (6160, "gelu"), (24_600, None)])
@pytest.mark.parametrize("m,k,group", [(5, 96, 32), (9, 1056, 32), (16, 2016, 96), (13, 2048, 128), (20, 96, 96),
                                       (17, 1056, 32), (32, 2016, 96), (31, 2048, 128)])
def test_more_rows_of_wide_layers(m, n, k, group, act):
    for kind in KINDS:
        run(m + k, m, n, k, group, kind, act, bias=m % 2 == 1)


@pytest.mark.parametrize("act", [None, "silu"])
def test_tiles_of_rows_beside_each_other(act):
    for kind in KINDS:
        run(5, 70, 2064, 1056, 32, kind, act, bias=True)


# ---------------------------------------------------------------- few tiles, two fragments a wave, a long K

@pytest.mark.parametrize("m", [1, 3, 4])
@pytest.mark.parametrize("k,group", [(4160, 32), (8352, 96), (10_240, 128), (12_448, 32)])
def test_few_rows_gated_of_a_long_k(m, k, group):
    for kind in KINDS:
        run(m + k, m, 40, k, group, kind, "silu", bias=True)


# The scales of more K than a workgroup keeps at a time: a second span after 3008 and 3808 (groups of 32, zero points,
# two fragments, 5 to 16 rows and more), 6208 (many tiles), three times that in groups of 96, four times of 128
@pytest.mark.parametrize("m", [5, 16, 17, 40])
@pytest.mark.parametrize("k,group", [(4192, 32), (7808, 32), (11_616, 96), (15_488, 128)])
def test_more_rows_of_a_k_of_several_spans(m, k, group):
    run(m + k, m, 40, k, group, KINDS[0], "silu", bias=True)
    run(m + k + 1, m, 40, k, group, KINDS[2], "gelu")


@pytest.mark.parametrize("m,k", [(11, 7200), (20, 4192)])
def test_more_rows_of_wide_layers_of_several_spans(m, k):
    run(m, m, 6160, k, 32, KINDS[0], "silu")


@pytest.mark.parametrize("m,k", [(11, 15_520), (20, 9760)])
def test_more_rows_of_one_fragment_of_several_spans(m, k):
    run(m, m, 40, k, 32, KINDS[0])


# ---------------------------------------------------------------- experts

# rows of the experts: one at most on average, three, nine and 25, on one expert more than all the others have
@pytest.mark.parametrize("experts,rows,most,n", [(48, 40, 17, 320), (24, 60, 30, 512), (24, 200, 90, 272),
                                                 (24, 600, 333, 272)])
@pytest.mark.parametrize("act", [None, "silu"])
def test_grouped_of_many_tiles_and_uneven_experts(experts, rows, most, n, act):
    k, group = 416, 32
    rng = np.random.default_rng([411, rows])
    splits = np.bincount(rng.integers(0, experts, rows - most), minlength=experts)
    splits[5] += most
    splits[[0, 7]] = 0
    total, per = int(splits.sum()) + 2, 2 * n if act else n
    for i, (fmt, dtype, scales, zeros) in enumerate(KINDS):
        w = Weights(40 + i, experts * per, k, group, fmt, scales, zeros)
        x = activations(3, total, k, dtype) * 0.25
        bias = activations(7, experts, per, dtype) if i == 0 else None
        d = torch.full((total, n), 55.0, dtype=DTYPES[dtype], device="cuda")
        m = torch.from_numpy(splits.astype(np.int32)).cuda()
        call = te().te_w4_grouped_gated_gemm if act else te().te_w4_grouped_gemm
        call(m, x, w.w, fmt, w.s, n, d, *([act] if act else []), zero=w.zero, bias=bias)
        at = 0
        for g, rows_g in enumerate(splits):
            if rows_g:
                check(f64(d)[at:at + rows_g], x[at:at + rows_g], w.rows(g * per, (g + 1) * per),
                      None if bias is None else f64(bias)[g], k, group, dtype, act, n)
            at += rows_g
        assert (f64(d)[at:] == 55.0).all()
