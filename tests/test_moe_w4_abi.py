"""CPU tests of the router's, the rows' and the 4-bit products' entry points: refusals of the C ABI (fake device
addresses, never dereferenced) and of the Python wrappers."""

import pytest
import torch

import mxfp8_mixed_precision_amd as te

L = te._lib
P, P2, P3, P4 = 0x10000, 0x20000, 0x30000, 0x40000
BAD = 0x10004
MOST = (1 << 31) - 65536


def route(score=te.TE_SCORE_SOFTMAX, logits=P, dt=te.TE_FP32, tokens=4, experts=8, topk=2, bias=None, normalize=1,
          scale=1.0, out=P2, weights=P3):
    return L.te_moe_route(score, logits, dt, tokens, experts, topk, bias, normalize, scale, out, weights, None)


def route_back(score=te.TE_SCORE_SOFTMAX, logits=P, dt=te.TE_FP32, tokens=4, experts=8, topk=2, normalize=1, scale=1.0,
               out=P2, weights=P3, dlogits=P4):
    return L.te_moe_route_backward(score, logits, dt, tokens, experts, topk, normalize, scale, out, weights, dlogits, None)


@pytest.mark.parametrize("call", [route, route_back])
def test_route_refusals(call):
    assert call(score=2) == te.TE_ERR_VALUE
    assert call(normalize=2) == te.TE_ERR_VALUE
    assert call(scale=float("nan")) == te.TE_ERR_VALUE
    assert call(scale=float("inf")) == te.TE_ERR_VALUE
    assert call(dt=te.TE_E4M3) == te.TE_ERR_DTYPE
    assert call(experts=0) == te.TE_ERR_SHAPE
    assert call(experts=1025) == te.TE_ERR_SHAPE
    assert call(topk=0) == te.TE_ERR_SHAPE
    assert call(topk=9) == te.TE_ERR_SHAPE
    assert call(experts=100, topk=65) == te.TE_ERR_SHAPE
    assert call(tokens=-1) == te.TE_ERR_SHAPE
    assert call(tokens=MOST) == te.TE_ERR_SHAPE                        # the slots pass 31 bits
    for k in ("logits", "out", "weights"):
        assert call(**{k: None}) == te.TE_ERR_NULL
    assert call(logits=BAD) == te.TE_ERR_ALIGN
    for k in ("out", "weights"):
        assert call(**{k: P + 2}) == te.TE_ERR_ALIGN
    assert call(tokens=0, logits=None, out=None, weights=None) == te.TE_OK


def test_route_own_refusals():
    assert route(bias=P + 2) == te.TE_ERR_ALIGN
    assert route_back(dlogits=None) == te.TE_ERR_NULL
    assert route_back(dlogits=BAD) == te.TE_ERR_ALIGN


def sort(experts=P, slots=100, n=8, splits=P2, row=P3, slot=P4, ws=None, ws_bytes=0):
    return L.te_moe_sort(experts, slots, n, splits, row, slot, ws, ws_bytes, None)


def test_sort_refusals():
    assert sort(n=0) == te.TE_ERR_SHAPE
    assert sort(n=1025) == te.TE_ERR_SHAPE
    assert sort(slots=-1) == te.TE_ERR_SHAPE
    assert sort(slots=MOST + 1) == te.TE_ERR_SHAPE
    for k in ("experts", "splits", "row", "slot"):
        assert sort(**{k: None}) == te.TE_ERR_NULL
        assert sort(**{k: P + 2}) == te.TE_ERR_ALIGN
    assert sort(slots=0, splits=None) == te.TE_ERR_NULL
    big, size = 1 << 20, te.te_moe_sort_workspace_size(1 << 20, 8)
    assert size > 0
    assert sort(slots=big) == te.TE_ERR_NULL
    assert sort(slots=big, ws=P + 2, ws_bytes=size) == te.TE_ERR_ALIGN
    assert sort(slots=big, ws=P, ws_bytes=size - 1) == te.TE_ERR_WORKSPACE


def test_sort_workspace_size():
    size = te.te_moe_sort_workspace_size
    assert size(0, 8) == size(-1, 8) == size(8, 0) == size(8, 1025) == size(MOST + 1, 8) == 0
    assert size(1, 8) == 0 and size(MOST, 1024) > 0
    for n in (1, 60, 1024):
        # a workspace of the largest call serves the smaller ones
        most = 0
        for slots in (1, 100, 5000, 1 << 17, 1 << 19, (1 << 19) + 1, 1 << 20, 1 << 24, MOST):
            most = max(most, size(slots, n))
            assert size(slots, n) % (4 * n) == 0
            assert size(slots, n) <= 4 * 256 * n
        assert most <= 4 * 256 * n


def test_sort_workspace_of_the_largest_batch_serves_every_smaller_one():
    size = te.te_moe_sort_workspace_size
    slots = sorted({s + d for s in (2048, 4096, 1 << 17, 1 << 19, 1 << 20, 3 << 19, 1 << 24, MOST - 1) for d in (-1, 0, 1)}
                   | set(range(1 << 18, 1 << 21, 30011)))
    for n in (1, 60, 1024):
        sizes = [size(s, n) for s in slots]
        assert sizes == sorted(sizes)
    for s in (100, 5000, 1 << 19, (1 << 19) + 1, MOST):
        assert [size(s, n) for n in (1, 8, 1024)] == sorted(size(s, n) for n in (1, 8, 1024))


def dispatch(x=P, dt=te.TE_BF16, tokens=4, cols=64, row=P2, topk=2, rows=8, y=P3, q=None, qs=None, qf=te.TE_E4M3):
    return L.te_moe_dispatch(x, dt, tokens, cols, row, topk, rows, y, q, qs, qf, None)


def combine(x=P, dt=te.TE_BF16, tokens=4, cols=64, row=P2, topk=2, rows=8, y=P3, w=P4):
    return L.te_moe_combine(x, dt, rows, cols, row, w, tokens, topk, y, None)


def combine_back(x=P, dt=te.TE_BF16, tokens=4, cols=64, row=P2, topk=2, rows=8, y=P3, w=P4, out=P, q=None, qs=None,
                 qf=te.TE_E5M2, dw=P2):
    return L.te_moe_combine_backward(x, out, dt, tokens, cols, row, w, topk, rows, y, q, qs, qf, dw, None)


@pytest.mark.parametrize("call", [dispatch, combine, combine_back])
def test_rows_refusals(call):
    assert call(dt=te.TE_E4M3) == te.TE_ERR_DTYPE
    assert call(topk=0) == te.TE_ERR_SHAPE
    assert call(topk=65) == te.TE_ERR_SHAPE
    assert call(tokens=-1) == te.TE_ERR_SHAPE
    assert call(tokens=MOST) == te.TE_ERR_SHAPE
    assert call(cols=-1) == te.TE_ERR_SHAPE
    assert call(cols=1 << 31) == te.TE_ERR_SHAPE
    assert call(rows=-1) == te.TE_ERR_SHAPE
    assert call(rows=1 << 31) == te.TE_ERR_SHAPE
    for k in ("x", "row", "y"):
        assert call(**{k: None}) == te.TE_ERR_NULL
    for k in ("x", "y"):
        assert call(**{k: BAD}) == te.TE_ERR_ALIGN
    assert call(row=P + 2) == te.TE_ERR_ALIGN


@pytest.mark.parametrize("call", [dispatch, combine_back])
def test_rows_mx_refusals(call):
    assert call(q=P) == te.TE_ERR_NULL
    assert call(qs=P) == te.TE_ERR_NULL
    assert call(q=P, qs=P2, dt=te.TE_FP16) == te.TE_ERR_DTYPE
    assert call(q=P, qs=P2, qf=te.TE_BF16) == te.TE_ERR_DTYPE
    assert call(q=P, qs=P2, cols=48) == te.TE_ERR_SHAPE
    assert call(q=BAD, qs=P2) == te.TE_ERR_ALIGN


def test_rows_empty_and_own_refusals():
    assert dispatch(tokens=0, x=None, row=None, y=None) == te.TE_OK
    assert dispatch(cols=0, x=None, row=None, y=None) == te.TE_OK
    assert dispatch(rows=0, x=None, row=None, y=None) == te.TE_OK
    assert combine(tokens=0, x=None, row=None, y=None) == te.TE_OK
    assert combine(cols=0, x=None, row=None, y=None) == te.TE_OK
    assert combine(w=P + 2) == te.TE_ERR_ALIGN
    assert combine_back(tokens=0, x=None, row=None, y=None, w=None, dw=None) == te.TE_OK
    assert combine_back(w=None) == te.TE_ERR_NULL
    assert combine_back(dw=None) == te.TE_ERR_NULL
    assert combine_back(out=None) == te.TE_ERR_NULL
    assert combine_back(dw=P + 2) == te.TE_ERR_ALIGN
    assert combine_back(out=BAD) == te.TE_ERR_ALIGN


def w4(x=P, dt=te.TE_BF16, w=P2, wf=te.TE_W4_INT4, s=P3, sdt=te.TE_BF16, z=None, group=32, M=3, N=20, K=64, d=P4,
       ddt=te.TE_BF16, bias=None):
    return L.te_w4_gemm(x, dt, w, wf, s, sdt, z, group, M, N, K, d, ddt, bias, None)


def w4_gated(x=P, dt=te.TE_BF16, w=P2, wf=te.TE_W4_INT4, s=P3, sdt=te.TE_BF16, z=None, group=32, M=3, N=20, K=64, d=P4,
             ddt=te.TE_BF16, bias=None, act=te.TE_ACT_SILU):
    return L.te_w4_gated_gemm(x, dt, w, wf, s, sdt, z, group, M, N, K, act, d, ddt, bias, None)


def w4_grouped(x=P, dt=te.TE_BF16, w=P2, wf=te.TE_W4_INT4, s=P3, sdt=te.TE_BF16, z=None, group=32, M=3, N=20, K=64,
               d=P4, ddt=te.TE_BF16, bias=None, G=2, splits=P):
    return L.te_w4_grouped_gemm(G, splits, M, x, dt, w, wf, s, sdt, z, group, N, K, d, ddt, bias, None)


def w4_grouped_gated(x=P, dt=te.TE_BF16, w=P2, wf=te.TE_W4_INT4, s=P3, sdt=te.TE_BF16, z=None, group=32, M=3, N=20,
                     K=64, d=P4, ddt=te.TE_BF16, bias=None, G=2, splits=P, act=te.TE_ACT_GELU):
    return L.te_w4_grouped_gated_gemm(G, splits, M, x, dt, w, wf, s, sdt, z, group, N, K, act, d, ddt, bias, None)


@pytest.mark.parametrize("call", [w4, w4_gated, w4_grouped, w4_grouped_gated])
def test_w4_refusals(call):
    assert call(wf=2) == te.TE_ERR_VALUE
    assert call(dt=te.TE_FP32, sdt=te.TE_FP32, ddt=te.TE_FP32) == te.TE_ERR_DTYPE
    assert call(sdt=te.TE_FP16) == te.TE_ERR_DTYPE
    assert call(sdt=te.TE_E4M3) == te.TE_ERR_DTYPE
    assert call(ddt=te.TE_FP16) == te.TE_ERR_DTYPE
    assert call(M=-1) == te.TE_ERR_SHAPE
    assert call(N=-1) == te.TE_ERR_SHAPE
    assert call(N=1 << 30) == te.TE_ERR_SHAPE
    assert call(N=(1 << 26) + 16) == te.TE_ERR_SHAPE
    assert call(K=(1 << 23) + 32) == te.TE_ERR_SHAPE
    assert call(group=0) == te.TE_ERR_SHAPE
    assert call(group=16) == te.TE_ERR_SHAPE
    assert call(group=48, K=96) == te.TE_ERR_SHAPE
    assert call(group=128) == te.TE_ERR_SHAPE                          # does not divide K
    assert call(wf=te.TE_W4_E2M1, z=P) == te.TE_ERR_NULL
    for k in ("x", "w", "s", "d"):
        assert call(**{k: None}) == te.TE_ERR_NULL
    for k in ("x", "w", "d"):
        assert call(**{k: BAD}) == te.TE_ERR_ALIGN
    assert call(s=P + 1) == te.TE_ERR_ALIGN
    assert call(s=P + 2, sdt=te.TE_FP32) == te.TE_ERR_ALIGN
    assert call(bias=P + 1) == te.TE_ERR_ALIGN
    assert call(M=0, x=None, d=None) == te.TE_OK


@pytest.mark.parametrize("call", [w4_gated, w4_grouped_gated])
def test_w4_gated_refusals(call):
    assert call(act=2) == te.TE_ERR_VALUE
    assert call(act=-1) == te.TE_ERR_VALUE


@pytest.mark.parametrize("call", [w4_grouped, w4_grouped_gated])
def test_w4_grouped_refusals(call):
    assert call(G=0) == te.TE_ERR_SHAPE
    assert call(G=1025) == te.TE_ERR_SHAPE
    assert call(N=0) == te.TE_ERR_SHAPE
    assert call(K=0) == te.TE_ERR_SHAPE
    assert call(splits=None) == te.TE_ERR_NULL
    assert call(splits=P + 2) == te.TE_ERR_ALIGN


def test_wrappers_refuse_wrong_tensors():
    l, e, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        te.te_moe_route("softmax", l, e, w)
    with pytest.raises(KeyError):
        te.te_moe_route("relu", l, e, w)
    with pytest.raises(ValueError, match="logits: expected"):
        te.te_moe_route("softmax", l.double(), e, w)
    with pytest.raises(ValueError, match="experts: expected int32"):
        te.te_moe_route("softmax", l, e.long(), w)
    with pytest.raises(ValueError, match="weights: expected shape"):
        te.te_moe_route("softmax", l, e, w[:3])
    with pytest.raises(ValueError, match="bias: expected"):
        te.te_moe_route("softmax", l, e, w, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="dlogits: expected"):
        te.te_moe_route_backward("softmax", l, e, w, l.half())
    s, m = torch.zeros(8, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="row_of: expected shape"):
        te.te_moe_sort(e, m, s, s)
    with pytest.raises(ValueError, match="m_splits"):
        te.te_moe_sort(e, None, e, s)
    x = torch.zeros(4, 48, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="y or q is required"):
        te.te_moe_dispatch(x, e)
    with pytest.raises(ValueError, match="cols % 32"):
        te.te_moe_dispatch(x, e, q=torch.zeros(8, 48, dtype=torch.uint8), q_scale=torch.zeros(8, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="y: expected shape"):
        te.te_moe_dispatch(x, e, y=torch.zeros(8, 47, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="row_of: expected shape"):
        te.te_moe_combine(torch.zeros(8, 48, dtype=torch.bfloat16), e[:3], x)
    with pytest.raises(ValueError, match="rows: expected shape"):
        te.te_moe_combine_backward(x, x, e, w, w, drows=torch.zeros(8, 48, dtype=torch.bfloat16))
    c, sc = torch.zeros(6, 32, dtype=torch.uint8), torch.zeros(6, 2, dtype=torch.bfloat16)
    x, d = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 6, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        te.te_w4_gemm(x, c, "int4", sc, d)
    with pytest.raises(KeyError):
        te.te_w4_gemm(x, c, "int3", sc, d)
    with pytest.raises(ValueError, match="w: expected shape"):
        te.te_w4_gemm(x, c[:, :16].contiguous(), "int4", sc, d)
    with pytest.raises(ValueError, match="do not divide"):
        te.te_w4_gemm(x, c, "int4", torch.zeros(6, 3, dtype=torch.bfloat16), d)
    with pytest.raises(ValueError, match="w_scale: expected"):
        te.te_w4_gemm(x, c, "int4", sc.half(), d)
    with pytest.raises(ValueError, match="d: expected"):
        te.te_w4_gemm(x, c, "int4", sc, d.half())
    with pytest.raises(ValueError, match="even number"):
        te.te_w4_gated_gemm(x, c[:5], "int4", sc[:5], d)
    with pytest.raises(ValueError, match="w: expected shape"):
        te.te_w4_grouped_gemm(m, x, c, "int4", sc, 6, d)
