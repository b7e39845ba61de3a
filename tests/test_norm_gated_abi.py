"""CPU tests of the norm and gated feed-forward entry points: refusals of the C ABI (fake device addresses, never
dereferenced) and of the Python wrappers."""

import pytest
import torch

import mxfp8_mixed_precision_amd as te

L = te._lib
P, P2, P3, P4 = 0x10000, 0x20000, 0x30000, 0x40000
BAD = 0x10004


def fwd(kind=te.TE_NORM_LAYER, x=P, dt=te.TE_BF16, rows=4, cols=64, res=None, gamma=P2, beta=None, wdt=te.TE_BF16,
        eps=1e-5, sum_out=None, y=P3, q=None, qs=None, qf=te.TE_E4M3, mean=None, rstd=None):
    return L.te_norm_forward(kind, x, dt, rows, cols, res, gamma, beta, wdt, eps, sum_out, y, q, qs, qf, mean, rstd,
                             None)


def test_norm_forward_refusals():
    assert fwd(kind=2) == te.TE_ERR_VALUE
    assert fwd(dt=te.TE_E4M3) == te.TE_ERR_DTYPE
    assert fwd(wdt=te.TE_FP16) == te.TE_ERR_DTYPE
    assert fwd(dt=te.TE_FP32, wdt=te.TE_BF16) == te.TE_ERR_DTYPE
    assert fwd(rows=-1) == te.TE_ERR_SHAPE
    assert fwd(cols=1 << 31) == te.TE_ERR_SHAPE
    assert fwd(eps=-1e-5) == te.TE_ERR_VALUE
    assert fwd(eps=float("nan")) == te.TE_ERR_VALUE
    assert fwd(eps=float("inf")) == te.TE_ERR_VALUE
    assert fwd(res=P) == te.TE_ERR_NULL                                # residual without sum_out
    assert fwd(sum_out=P) == te.TE_ERR_NULL
    assert fwd(q=P) == te.TE_ERR_NULL
    assert fwd(mean=P) == te.TE_ERR_NULL                               # mean without rstd
    assert fwd(rstd=P) == te.TE_ERR_NULL
    assert fwd(kind=te.TE_NORM_RMS, beta=P) == te.TE_ERR_NULL
    assert fwd(kind=te.TE_NORM_RMS, mean=P, rstd=P) == te.TE_ERR_NULL
    assert fwd(dt=te.TE_FP16, wdt=te.TE_FP16, q=P, qs=P2) == te.TE_ERR_DTYPE
    assert fwd(q=P, qs=P2, qf=te.TE_BF16) == te.TE_ERR_DTYPE
    assert fwd(q=P, qs=P2, cols=48) == te.TE_ERR_SHAPE
    assert fwd(x=None) == te.TE_ERR_NULL
    assert fwd(gamma=None) == te.TE_ERR_NULL
    assert fwd(y=None) == te.TE_ERR_NULL
    for k in ("x", "gamma", "beta", "y"):
        assert fwd(**{k: BAD}) == te.TE_ERR_ALIGN
    assert fwd(res=BAD, sum_out=P) == te.TE_ERR_ALIGN
    assert fwd(mean=P + 2, rstd=P) == te.TE_ERR_ALIGN
    assert fwd(rows=0, x=None, gamma=None, y=None) == te.TE_OK
    assert fwd(cols=0, x=None, gamma=None, y=None) == te.TE_OK


def bwd(kind=te.TE_NORM_LAYER, dy=P, x=P2, dskip=None, dt=te.TE_BF16, rows=4, cols=64, gamma=P3, wdt=te.TE_BF16,
        mean=P, rstd=P, dx=P4, dg=P4, db=P4, ws=P, ws_bytes=1 << 30):
    return L.te_norm_backward(kind, dy, x, dskip, dt, rows, cols, gamma, wdt, mean, rstd, dx, dg, db, ws, ws_bytes,
                              None)


def test_norm_backward_refusals():
    assert bwd(kind=-1) == te.TE_ERR_VALUE
    assert bwd(dt=te.TE_E8M0) == te.TE_ERR_DTYPE
    assert bwd(wdt=te.TE_FP16) == te.TE_ERR_DTYPE
    assert bwd(rows=-4) == te.TE_ERR_SHAPE
    assert bwd(kind=te.TE_NORM_RMS, mean=None) == te.TE_ERR_NULL       # dbeta with RMS norm
    assert bwd(kind=te.TE_NORM_RMS, db=None) == te.TE_ERR_NULL         # mean with RMS norm
    for k in ("dy", "x", "gamma", "mean", "rstd", "dx", "dg", "ws"):
        assert bwd(**{k: None}) == te.TE_ERR_NULL
    for k in ("dy", "x", "dskip", "gamma", "dx", "dg", "db", "ws"):
        assert bwd(**{k: BAD}) == te.TE_ERR_ALIGN
    assert bwd(ws_bytes=te.te_norm_backward_workspace_size(4, 64) - 1) == te.TE_ERR_WORKSPACE
    assert bwd(cols=0, dy=None, x=None, gamma=None, dg=None, db=None, dx=None, ws=None) == te.TE_OK


def test_norm_backward_workspace_size():
    assert te.te_norm_backward_workspace_size(0, 64) == 0
    assert te.te_norm_backward_workspace_size(64, 0) == 0
    assert te.te_norm_backward_workspace_size(-1, 64) == 0
    for rows, cols in ((1, 1), (100, 77), (5000, 4096), (1 << 20, 70001)):
        size = te.te_norm_backward_workspace_size(rows, cols)
        assert size >= 2 * 4 * cols and size % (8 * cols) == 0         # whole rows of both gradients' partial sums


def gated(a=P, sa=P2, fa=te.TE_E4M3, b=P, sb=P2, fb=te.TE_E4M3, M=3, N=64, K=256, act=te.TE_ACT_SILU, d=P3, ds=None,
          dt=te.TE_BF16, bias=None, aux=None):
    return L.te_mxfp8_gated_gemm(a, sa, fa, b, sb, fb, M, N, K, act, d, ds, dt, bias, aux, None, 0, None)


def dgated(a=P, sa=P2, fa=te.TE_E5M2, b=P, sb=P2, fb=te.TE_E4M3, M=3, N=64, K=256, act=te.TE_ACT_GELU, aux=P4, d=P3):
    return L.te_mxfp8_dgated_gemm(a, sa, fa, b, sb, fb, M, N, K, act, aux, d, None, 0, None)


@pytest.mark.parametrize("call", [gated, dgated])
def test_gated_refusals(call):
    assert call(act=2) == te.TE_ERR_VALUE
    assert call(fa=te.TE_BF16) == te.TE_ERR_DTYPE
    assert call(fa=te.TE_E5M2, fb=te.TE_E5M2) == te.TE_ERR_DTYPE
    assert call(M=-1) == te.TE_ERR_SHAPE
    assert call(N=24) == te.TE_ERR_SHAPE
    assert call(K=64) == te.TE_ERR_SHAPE
    assert call(K=(1 << 23) + 128) == te.TE_ERR_SHAPE
    assert call(N=1 << 30) == te.TE_ERR_SHAPE
    assert call(N=1 << 20, K=1 << 16) == te.TE_ERR_SHAPE              # the weights' scales pass 32-bit offsets
    for k in ("a", "sa", "b", "sb", "d"):
        assert call(**{k: None}) == te.TE_ERR_NULL
    for k in ("a", "b", "d", "aux"):
        assert call(**{k: BAD}) == te.TE_ERR_ALIGN
    assert call(sa=P + 2) == te.TE_ERR_ALIGN
    assert call(M=0, a=None, sa=None, d=None) == te.TE_OK
    assert call(N=0, b=None, sb=None, d=None) == te.TE_OK


def test_gated_output_refusals():
    assert gated(dt=te.TE_FP32) == te.TE_ERR_DTYPE
    assert gated(ds=P) == te.TE_ERR_NULL                               # a bf16 D has no scales
    assert gated(dt=te.TE_E4M3) == te.TE_ERR_NULL                      # an MXFP8 D needs them
    assert gated(dt=te.TE_E4M3, ds=P, N=48) == te.TE_ERR_SHAPE
    assert gated(bias=P + 2) == te.TE_ERR_ALIGN
    assert dgated(aux=None) == te.TE_ERR_NULL


def grouped(G=2, splits=P, M=5, N=64, K=256, d=P3, a=P, aux=None):
    return L.te_mxfp8_grouped_gated_gemm(G, splits, M, a, P2, te.TE_E4M3, P, P2, te.TE_E4M3, N, K, te.TE_ACT_SILU, d,
                                         None, aux, None)


def grouped_back(G=2, splits=P, M=5, N=64, K=256, d=P3, a=P, aux=P4):
    return L.te_mxfp8_grouped_dgated_gemm(G, splits, M, a, P2, te.TE_E4M3, P, P2, te.TE_E4M3, N, K, te.TE_ACT_SILU,
                                          aux, d, None)


@pytest.mark.parametrize("call", [grouped, grouped_back])
def test_grouped_gated_refusals(call):
    assert call(G=0) == te.TE_ERR_SHAPE
    assert call(G=1025) == te.TE_ERR_SHAPE
    assert call(N=0) == te.TE_ERR_SHAPE
    assert call(K=0) == te.TE_ERR_SHAPE
    assert call(N=24) == te.TE_ERR_SHAPE
    assert call(M=-1) == te.TE_ERR_SHAPE
    assert call(splits=None) == te.TE_ERR_NULL
    assert call(splits=P + 2) == te.TE_ERR_ALIGN
    assert call(d=None) == te.TE_ERR_NULL
    assert call(a=BAD) == te.TE_ERR_ALIGN
    assert call(M=0, d=None, a=None) == te.TE_OK


def test_wrappers_refuse_wrong_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    g = torch.ones(64, dtype=torch.bfloat16)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU tensor"):
        te.te_norm_forward("layer", x, g, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="gamma"):
        te.te_norm_forward("layer", x, g.half(), y=x)
    with pytest.raises(ValueError, match="2-D"):
        te.te_norm_forward("layer", x[0], g, y=x[0])
    with pytest.raises(ValueError, match="x: expected"):
        te.te_norm_forward("layer", x.double(), g, y=x)
    with pytest.raises(ValueError, match="cols % 32"):
        te.te_norm_forward("layer", x[:, :40].contiguous(), g[:40], q=f, q_scale=f)
    with pytest.raises(KeyError):
        te.te_norm_forward("batch", x, g, y=x)
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8)
    b, bs = torch.zeros(33, 256, dtype=torch.uint8), torch.zeros(33, 8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="even number"):
        te.te_mxfp8_gated_gemm(q, s, "e4m3", b, bs, "e4m3", None)
    with pytest.raises(ValueError, match="a is required"):
        te.te_mxfp8_dgated_gemm(None, s, "e4m3", b, bs, "e4m3", None, None)
    with pytest.raises(ValueError, match="m_splits"):
        te.te_mxfp8_grouped_gated_gemm(None, q, s, "e4m3", b, bs, "e4m3", 16, None)


@pytest.mark.parametrize("cols", [1, 16, 130, 1024, 2048, 2056, 5120, 5128, 8192, 8200, 16384, 16392, 70001])
def test_norm_backward_workspace_of_a_batch_serves_smaller_ones(cols):
    """A program that sizes its workspace for its longest batch has enough for every shorter one."""
    rows = sorted({r + d for e in range(21) for r in (1 << e,) for d in (-1, 0, 1)} - {0})
    sizes = [te.te_norm_backward_workspace_size(r, cols) for r in rows]
    assert sizes == sorted(sizes)
    assert bwd(rows=rows[5], cols=cols, ws_bytes=sizes[5] - 1) == te.TE_ERR_WORKSPACE


@pytest.mark.parametrize("rows", [1, 37, 255, 511, 1023, 2047, 4096, 16384, 1 << 20])
def test_norm_backward_workspace_of_the_widest_norm_serves_narrower_ones(rows):
    cols = sorted({8 * nt + d for nt in (16, 32, 64, 128, 192, 256, 512, 640, 768, 1024, 2048, 4096)
                   for d in (-8, -1, 0, 1, 8)})
    sizes = [te.te_norm_backward_workspace_size(rows, c) for c in cols]
    assert sizes == sorted(sizes)


def test_norm_backward_workspace_holds_the_partial_sums_of_every_batch():
    """Never less than one row of both gradients' sums, and bounded: two for each CU, or those of 16384 columns."""
    for rows in (1, 100, 5000, 1 << 20):
        for cols in (1, 77, 4096, 16384, 16385, 70001):
            size = te.te_norm_backward_workspace_size(rows, cols)
            assert 8 * cols <= size <= 8 * 512 * max(cols, 16384)
