"""The norm and gated operators as a LayerNormMLP block uses them: a whole forward and backward pass, captured and
replayed, on other streams, with guarded outputs, shared inputs and sizes past 32-bit offsets."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_to_f64, host

pytestmark = pytest.mark.gpu

U8 = dict(dtype=torch.uint8, device="cuda")
BF = dict(dtype=torch.bfloat16, device="cuda")


def te():
    import mxfp8_mixed_precision_amd as m
    return m


def randn(seed, *shape, sigma=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sigma).bfloat16()


class Block:
    """norm(x + residual) -> gated projection -> down projection, MXFP8 throughout, with its backward pass."""

    def __init__(self, tokens, hidden, ffn, act="silu", kind="layer"):
        m = te()
        self.T, self.H, self.F, self.act, self.kind = tokens, hidden, ffn, act, kind
        self.x, self.res, self.dout = randn(1, tokens, hidden), randn(2, tokens, hidden), randn(3, tokens, hidden)
        self.gamma = (1 + 0.1 * randn(4, hidden).float()).bfloat16()
        self.beta = randn(5, hidden, sigma=0.1) if kind == "layer" else None
        self.w1, self.w2 = randn(6, 2 * ffn, hidden, sigma=0.05), randn(7, hidden, ffn, sigma=0.05)
        self.b1 = randn(8, 2 * ffn, sigma=0.1)
        # both weights' operands: along the contracted dimension forward, transposed backward
        self.q1, self.s1, self.q1t, self.s1t = m.mxfp8_quantize(self.w1, "e4m3", "both")
        self.q2, self.s2, self.q2t, self.s2t = m.mxfp8_quantize(self.w2, "e4m3", "both")

    def run(self, stream=None):
        m, k = te(), dict(stream=stream)
        o = {}
        # forward
        o["y"], o["q"], o["qs"], o["sum"], o["mean"], o["rstd"] = m.norm_forward(
            self.kind, self.x, self.gamma, self.beta, 1e-5, self.res, "e4m3", **k)
        o["h"], _, o["aux"] = m.mxfp8_gated_gemm(o["q"], o["qs"], "e4m3", self.q1, self.s1, "e4m3", self.act, self.b1,
                                                 want_aux=True, **k)
        hq, hs, _, _ = m.mxfp8_quantize(o["h"], "e4m3", "row", **k)
        o["out"], _ = m.mxfp8_gemm(hq, hs, "e4m3", self.q2, self.s2, "e4m3", **k)
        # backward
        dq, dqs, _, _ = m.mxfp8_quantize(self.dout, "e5m2", "row", **k)
        o["dq"], o["dqs"] = dq, dqs
        o["dp"] = m.mxfp8_dgated_gemm(dq, dqs, "e5m2", self.q2t, self.s2t, "e4m3", o["aux"], self.act, **k)
        pq, ps, pqt, pst, o["db1"] = m.mxfp8_quantize_bgrad(o["dp"], "e5m2", **k)
        _, _, yqt, yst = m.mxfp8_quantize(o["y"], "e4m3", "col", **k)
        o["dw1"], _ = m.mxfp8_gemm(pqt, pst, "e5m2", yqt, yst, "e4m3", **k)
        o["dy"], _ = m.mxfp8_gemm(pq, ps, "e5m2", self.q1t, self.s1t, "e4m3", **k)
        o["dx"], o["dgamma"], o["dbeta"] = m.norm_backward(self.kind, o["dy"], o["sum"], self.gamma, o["mean"],
                                                           o["rstd"], dskip=self.dout, **k)
        return {n: v for n, v in o.items() if v is not None}


@pytest.mark.parametrize("kind,act", [("layer", "silu"), ("rms", "gelu")])
def test_block_against_the_definitions_in_64_bits(kind, act):
    """Each stage of the run against the oracle on that stage's own inputs.  Relative 2-norm errors: a bf16 result is
    rounded by at most 2^-8 of each value; the products' errors (the scaled MFMA's truncation, 2^-13 of a group's
    largest product at most for each, random in sign) and the fp32 arithmetic stay below another 2^-8 in the norm."""
    b = Block(256, 256, 384, act, kind)
    o = b.run()
    torch.cuda.synchronize()

    def f(t):
        return bf16_to_f64(host(t)) if t.dtype == torch.bfloat16 else t.cpu().double().numpy()

    def near(got, want):
        assert np.linalg.norm(f(got) - want) <= 2.0 ** -7 * np.linalg.norm(want)

    deq = lambda q, s, fmt: oracle.dequantize(host(q), host(s), fmt)  # noqa: E731
    s = f(o["sum"])
    y, mean, rstd = oracle.norm_forward(s, f(b.gamma), None if b.beta is None else f(b.beta), 1e-5, kind)
    near(o["y"], y)
    p = deq(o["q"], o["qs"], oracle.E4M3) @ deq(b.q1, b.s1, oracle.E4M3).T + f(b.b1)
    near(o["aux"], p)
    near(o["h"], oracle.gated(p, act))
    dh = deq(o["dq"], o["dqs"], oracle.E5M2) @ deq(b.q2t, b.s2t, oracle.E4M3).T
    near(o["dp"], oracle.gated_grad(dh, f(o["aux"]), act))
    mean64 = f(o["mean"]) if kind == "layer" else None
    dx, dgamma, dbeta = oracle.norm_backward(f(o["dy"]), s, f(b.gamma), mean64, f(o["rstd"]), kind, f(b.dout))
    near(o["dx"], dx)
    near(o["dgamma"], dgamma)
    if kind == "layer":
        near(o["dbeta"], dbeta)
    near(o["db1"], f(o["dp"]).sum(0))


@pytest.mark.parametrize("tokens,hidden,ffn", [(128, 256, 384), (4096, 2048, 4096)])
def test_block_captured_and_replayed(tokens, hidden, ffn):
    """Replays with eager work in between, against eager runs; the larger one takes the 4-wave kernel and its workspace."""
    b = Block(tokens, hidden, ffn)
    want = b.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b.run()
    for replay in range(4):
        for v in got.values():
            v.zero_()
        if replay == 2:  # other inputs in the same buffers
            b.x.copy_(randn(50, tokens, hidden))
            want = b.run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, v in got.items():
            assert torch.equal(v, want[n]), f"replay {replay}: {n}"


def test_two_streams_at_once():
    blocks = [Block(384, 512, 512), Block(256, 512, 640, "gelu", "rms")]
    want = [b.run() for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        got = [b.run(stream=s) for b, s in zip(blocks, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(g[n], w[n]) for n in w)


class Guarded:
    """A tensor inside a larger buffer whose other bytes are watched."""

    def __init__(self, shape, dtype, init=None):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((n + 512,), 0xA5, **U8)
        self.t = self.raw[256:256 + n].view(dtype).view(shape)
        self.n = n
        if init is not None:
            self.t.copy_(init)

    def intact(self):
        return bool((self.raw[:256] == 0xA5).all() and (self.raw[256 + self.n:] == 0xA5).all())


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 33), (2, 1001), (17, 130), (1, 4099), (3, 9001), (2, 33001)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_norms_write_only_their_outputs(rows, cols, dt):
    m = te()
    x, res = torch.randn(rows, cols, device="cuda").to(dt), torch.randn(rows, cols, device="cuda").to(dt)
    gamma = torch.ones(cols, device="cuda").to(dt)
    full = {n: Guarded((rows, cols), dt) for n in ("y", "sum", "dx")}
    stat = {n: Guarded((rows,), torch.float32) for n in ("mean", "rstd")}
    grad = {n: Guarded((cols,), dt) for n in ("dgamma", "dbeta")}
    ws = Guarded((m.te_norm_backward_workspace_size(rows, cols),), torch.uint8)
    m.te_norm_forward("layer", x, gamma, gamma, 1e-5, y=full["y"].t, residual=res, sum_out=full["sum"].t,
                      mean=stat["mean"].t, rstd=stat["rstd"].t)
    m.te_norm_backward("layer", res, full["sum"].t, gamma, stat["mean"].t, stat["rstd"].t, full["dx"].t,
                       grad["dgamma"].t, grad["dbeta"].t, workspace=ws.t)
    torch.cuda.synchronize()
    for gr in (full, stat, grad, {"workspace": ws}):
        for n, v in gr.items():
            assert v.intact(), n


@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (5, 48, 256), (33, 32, 384), (70, 80, 128), (130, 144, 256),
                                   (1290, 4128, 128)])
def test_gated_gemms_write_only_their_outputs(M, N, K):
    m = te()
    a, sa, _, _ = m.mxfp8_quantize(randn(1, M, K))
    b, sb, _, _ = m.mxfp8_quantize(randn(2, 2 * N, K))
    d, aux, grad = Guarded((M, N), torch.bfloat16), Guarded((M, 2 * N), torch.bfloat16), \
        Guarded((M, 2 * N), torch.bfloat16)
    m.te_mxfp8_gated_gemm(a, sa, "e4m3", b, sb, "e4m3", d.t, aux=aux.t)
    m.te_mxfp8_dgated_gemm(a, sa, "e4m3", b[:N], sb[:N], "e4m3", aux.t, grad.t)
    outs = [d, aux, grad]
    if N % 32 == 0:
        q, s = Guarded((M, N), torch.uint8), Guarded((M, N // 32), torch.uint8)
        m.te_mxfp8_gated_gemm(a, sa, "e4m3", b, sb, "e4m3", q.t, d_scale=s.t, d_fmt="e4m3")
        outs += [q, s]
    torch.cuda.synchronize()
    assert all(o.intact() for o in outs)


def test_one_tensor_given_twice():
    m = te()
    x = randn(1, 9, 300)
    g = randn(2, 300)
    y, _, _, total, mean, rstd = m.norm_forward("layer", x, g, g, residual=x)
    assert torch.equal(total, (x.float() * 2).bfloat16())
    again = m.norm_forward("layer", total, g, g.clone())
    assert torch.equal(again[0], y)
    same = m.norm_backward("layer", x, x, g, mean, rstd, dskip=x)
    other = m.norm_backward("layer", x.clone(), x.clone(), g, mean, rstd, dskip=x.clone())
    assert all(torch.equal(p, q) for p, q in zip(same, other))
    a, sa, _, _ = m.mxfp8_quantize(randn(3, 32, 128))
    d1 = m.mxfp8_gated_gemm(a, sa, "e4m3", a, sa, "e4m3")[0]
    d2 = m.mxfp8_gated_gemm(a, sa, "e4m3", a.clone(), sa.clone(), "e4m3")[0]
    assert torch.equal(d1, d2)


def test_norms_past_32_bit_offsets():
    rows, cols = 70_000, 32_768  # 2.3e9 elements
    m = te()
    x = torch.empty((rows, cols), **BF)
    x[:4], x[-4:] = randn(1, 4, cols), randn(2, 4, cols)
    x[4:-4] = 1.0
    gamma = randn(3, cols)
    y, _, _, _, _, rstd = m.norm_forward("rms", x, gamma)
    for sl in (slice(0, 4), slice(rows - 4, rows)):
        want = m.norm_forward("rms", x[sl].clone(), gamma)
        assert torch.equal(y[sl], want[0]) and torch.equal(rstd[sl], want[5])
    del y
    dx, dgamma, _ = m.norm_backward("rms", x, x, gamma, None, rstd)
    want = m.norm_backward("rms", x[-4:].clone(), x[-4:].clone(), gamma, None, rstd[-4:].clone())
    assert torch.equal(dx[-4:], want[0])
    assert torch.isfinite(dgamma.float()).all()
    del x, dx
    torch.cuda.empty_cache()


def test_norm_backward_of_a_row_longer_than_one_launch_of_columns():
    cols = 2 ** 26 + 40
    m = te()
    x, dy = randn(1, 1, 1024).repeat(1, 65_537)[:, :cols].contiguous(), torch.ones((1, cols), **BF)
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    _, dgamma, dbeta = m.norm_backward("layer", dy, x, torch.ones(cols, **BF), mean, rstd)
    assert torch.equal(dgamma, x[0]) and torch.equal(dbeta, dy[0])  # one row: dy xh and dy themselves
    del x, dy, dgamma, dbeta
    torch.cuda.empty_cache()


def test_gated_gemms_past_32_bit_offsets():
    M, N, K = 140_100, 8_192, 128  # 2.3e9 pre-activations
    m = te()
    a, sa, _, _ = m.mxfp8_quantize(randn(1, M, K))
    b, sb, _, _ = m.mxfp8_quantize(randn(2, 2 * N, K))
    d, _, aux = m.mxfp8_gated_gemm(a, sa, "e4m3", b, sb, "e4m3", want_aux=True)
    tail = [t[-100:].clone() for t in (a, sa)]
    want = m.mxfp8_gated_gemm(*tail, "e4m3", b, sb, "e4m3", want_aux=True)
    assert torch.equal(d[-100:], want[0]) and torch.equal(aux[-100:], want[2])
    grad = m.mxfp8_dgated_gemm(a, sa, "e4m3", b[:N], sb[:N], "e4m3", aux)
    assert torch.equal(grad[-100:], m.mxfp8_dgated_gemm(*tail, "e4m3", b[:N], sb[:N], "e4m3", want[2]))
    del d, aux, grad
    torch.cuda.empty_cache()


def test_gpu_refusals():
    m = te()
    x, g = randn(1, 8, 64), randn(2, 64)
    with pytest.raises(ValueError, match="contiguous"):
        m.te_norm_forward("layer", randn(1, 64, 8).t(), g, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="shape"):
        m.te_norm_forward("layer", x, g[:60], y=torch.empty_like(x))
    with pytest.raises(ValueError, match="device"):
        m.te_norm_forward("layer", x, g.cpu(), y=torch.empty_like(x))
    with pytest.raises(m.TemxError, match="TE_ERR_ALIGN"):
        raw = torch.empty(8 * 64 + 8, **BF)
        m.te_norm_forward("layer", x, g, y=raw[1:1 + 8 * 64].view(8, 64))
    r = torch.ones(8, device="cuda")
    with pytest.raises(m.TemxError, match="TE_ERR_WORKSPACE"):
        m.te_norm_backward("rms", x, x, g, None, r, torch.empty_like(x), torch.empty_like(g),
                           workspace=torch.empty(16, **U8))
    with pytest.raises(m.TemxError, match="TE_ERR_NULL"):
        m.te_norm_backward("rms", x, x, g, None, r, torch.empty_like(x), torch.empty_like(g))
    a, sa, _, _ = m.mxfp8_quantize(randn(3, 4, 128))
    b, sb, _, _ = m.mxfp8_quantize(randn(4, 96, 128))
    with pytest.raises(m.TemxError, match="TE_ERR_DTYPE"):
        m.mxfp8_gated_gemm(a, sa, "e5m2", b, sb, "e5m2")
    with pytest.raises(m.TemxError, match="TE_ERR_SHAPE"):
        m.mxfp8_gated_gemm(a, sa, "e4m3", b, sb, "e4m3", out_fmt="e4m3")  # N = 48


def test_streams_given_as_handles():
    b = Block(128 * 32, 256, 384)  # (the weight gradient contracts over the tokens: whole 128s)
    want = b.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side.cuda_stream, torch.cuda.current_stream().cuda_stream, 0):
        got = b.run(stream=handle)
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want), handle
