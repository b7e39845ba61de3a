"""The router, the sort, the experts' rows and the experts' GEMMs as a mixture-of-experts block uses them: a whole forward
and backward pass, a decoding step on 4-bit weights, captured and replayed, on other streams, past 32-bit offsets."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_to_f64, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def te():
    import mxfp8_mixed_precision_amd as m
    return m


def randn(seed, *shape, sigma=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sigma).bfloat16()


def f(t):
    return bf16_to_f64(host(t)) if t.dtype == torch.bfloat16 else t.cpu().double().numpy()


def near(got, want, rel):
    assert np.linalg.norm(f(got) - want) <= rel * np.linalg.norm(want)


class Block:
    """Router -> experts' rows as MXFP8 -> gated projection -> down projection -> combine, with its backward pass."""

    def __init__(self, tokens, hidden, ffn, experts, topk, score="softmax", seed=0):
        m = te()
        self.T, self.H, self.F, self.E, self.K, self.score = tokens, hidden, ffn, experts, topk, score
        self.x, self.dy = randn(seed + 1, tokens, hidden), randn(seed + 2, tokens, hidden)
        self.logits = randn(seed + 3, tokens, experts).float()
        self.bias = randn(seed + 4, experts, sigma=0.05).float()
        w1, w2 = randn(seed + 5, experts * 2 * ffn, hidden, sigma=0.05), randn(seed + 6, experts * hidden, ffn, sigma=0.05)
        self.w1, self.w2 = w1, w2
        self.q1, self.s1, _, _ = m.mxfp8_quantize(w1, "e4m3", "row")
        self.q2, self.s2, _, _ = m.mxfp8_quantize(w2, "e4m3", "row")
        # the transposed copies of the backward, an expert at a time
        turn = lambda w, r: w.view(experts, r, -1).transpose(1, 2).contiguous().view(-1, r)  # noqa: E731
        self.q1t, self.s1t, _, _ = m.mxfp8_quantize(turn(w1, 2 * ffn), "e4m3", "row")
        self.q2t, self.s2t, _, _ = m.mxfp8_quantize(turn(w2, hidden), "e4m3", "row")

    def run(self, stream=None):
        m, k, o = te(), dict(stream=stream), {}
        R = self.T * self.K
        o["experts"], o["weights"] = m.moe_route(self.score, self.logits, self.K, self.bias, True, 1.5, **k)
        o["splits"], o["row_of"], o["slot_of"] = m.moe_sort(o["experts"], self.E, **k)
        _, o["q"], o["qs"] = m.moe_dispatch(self.x, o["row_of"], "e4m3", want_y=False, **k)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            o["h"] = torch.empty((R, self.F), dtype=torch.bfloat16, device="cuda")
            o["aux"] = torch.empty((R, 2 * self.F), dtype=torch.bfloat16, device="cuda")
            o["dp"] = torch.empty((R, 2 * self.F), dtype=torch.bfloat16, device="cuda")
        m.te_mxfp8_grouped_gated_gemm(o["splits"], o["q"], o["qs"], "e4m3", self.q1, self.s1, "e4m3", self.F, o["h"],
                                      "silu", None, o["aux"], stream)
        hq, hs, _, _ = m.mxfp8_quantize(o["h"], "e4m3", "row", **k)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            o["rows"], _ = m.mxfp8_grouped_gemm(o["splits"], hq, hs, "e4m3", self.q2, self.s2, "e4m3", self.H, **k)
        o["y"] = m.moe_combine(o["rows"], o["row_of"], o["weights"], **k)
        # backward
        _, o["dweights"], o["dq"], o["dqs"] = m.moe_combine_backward(self.dy, o["rows"], o["row_of"], o["weights"],
                                                                     "e5m2", want_drows=False, **k)
        m.te_mxfp8_grouped_dgated_gemm(o["splits"], o["dq"], o["dqs"], "e5m2", self.q2t, self.s2t, "e4m3", self.F,
                                       o["aux"], o["dp"], "silu", stream)
        pq, ps, _, _ = m.mxfp8_quantize(o["dp"], "e5m2", "row", **k)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            o["drows"], _ = m.mxfp8_grouped_gemm(o["splits"], pq, ps, "e5m2", self.q1t, self.s1t, "e4m3", self.H, **k)
        o["dx"] = m.moe_combine(o["drows"], o["row_of"], **k)
        o["dlogits"] = m.moe_route_backward(self.score, self.logits, o["experts"], o["dweights"], True, 1.5, **k)
        return o


@pytest.mark.parametrize("score,topk", [("softmax", 2), ("sigmoid", 5)])
def test_block_against_the_definitions_in_64_bits(score, topk):
    """Each stage of the run against the oracle on that stage's own inputs, in relative 2-norms: bf16 results are rounded
    by at most 2^-8 of each value; fp32 ones by a few hundred roundings of 2^-24."""
    b = Block(150, 256, 128, 16, topk, score)
    o = b.run()
    torch.cuda.synchronize()
    e, w = oracle.route(f(b.logits), topk, score, f(b.bias), True, 1.5)
    assert np.array_equal(host(o["experts"]), e)
    near(o["weights"], w, 300 * U)
    splits, row_of, slot_of = oracle.sort_slots(e, b.E)
    assert np.array_equal(host(o["splits"]), splits) and np.array_equal(host(o["slot_of"]), slot_of)
    assert np.array_equal(host(o["row_of"]).reshape(-1), row_of)
    row_of = row_of.reshape(e.shape)
    qx, sx, _, _ = te().mxfp8_quantize(b.x, "e4m3", "row")
    assert np.array_equal(host(o["q"]), host(qx)[slot_of // topk])
    assert np.array_equal(host(o["qs"]), host(sx)[slot_of // topk])
    near(o["y"], oracle.combine(f(o["rows"]), row_of, f(o["weights"])), 2.0 ** -8)
    drows, dweights = oracle.combine_backward(f(b.dy), f(o["rows"]), row_of, f(o["weights"]))
    near(o["dweights"], dweights, 300 * U)
    codes, scales = oracle.quantize_rowwise(host(torch.from_numpy(drows.astype(np.float32)).bfloat16()), oracle.E5M2)
    assert (host(o["dq"]) != codes).mean() < 1e-3 and (host(o["dqs"]) != scales).mean() < 1e-3  # float64's own rounding to bf16
    near(o["dx"], oracle.combine(f(o["drows"]), row_of), 2.0 ** -8)
    near(o["dlogits"], oracle.route_backward(f(b.logits), e, f(o["dweights"]), score, True, 1.5), 300 * U)


def test_block_whole_against_the_definition_on_the_operands_values():
    """The run end to end in float64 on the values that the MXFP8 operands stand for, the hidden values rounded to bf16 and
    quantized as the block does.  Off by at most 2^-8 of the norm each: the hidden values that another rounding to bf16
    moves (and their codes with them, the fewer), the experts' rows, and y; the scaled MFMA's truncation, 2^-13 of a
    group's largest product, stays below another 2^-8."""
    b = Block(128, 256, 128, 16, 2)
    o = b.run()
    torch.cuda.synchronize()
    e = host(o["experts"])
    value = lambda q, s: oracle.dequantize(host(q), host(s), oracle.E4M3)  # noqa: E731
    w1, w2 = value(b.q1, b.s1).reshape(16, 256, 256), value(b.q2, b.s2).reshape(16, 256, 128)
    qx, sx, _, _ = te().mxfp8_quantize(b.x, "e4m3", "row")
    x, w, want = value(qx, sx), f(o["weights"]), np.zeros((128, 256))
    for t, k in np.ndindex(e.shape):
        p = x[t] @ w1[e[t, k]].T
        h = torch.from_numpy((oracle.activation(p[:128], "silu") * p[128:]).astype(np.float32)).bfloat16()
        codes, scales = oracle.quantize_rowwise(host(h)[None], oracle.E4M3)
        want[t] += w[t, k] * (w2[e[t, k]] @ oracle.dequantize(codes, scales, oracle.E4M3)[0])
    near(o["y"], want, 4 * 2.0 ** -8)


def same(a, b):
    assert a.keys() == b.keys()
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


def test_block_captured_and_replayed():
    b = Block(100, 256, 128, 16, 3)
    want = {n: v.clone() for n, v in b.run().items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.run()
    for i in range(4):
        for v in out.values():
            v.zero_()
        other = b.run()                                                # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        same(out, want)
        same(other, want)
    # new inputs in the captured buffers
    c = Block(100, 256, 128, 16, 3, seed=50)
    for n in ("x", "dy", "logits", "bias", "q1", "s1", "q2", "s2", "q1t", "s1t", "q2t", "s2t"):
        getattr(b, n).copy_(getattr(c, n))
    g.replay()
    torch.cuda.synchronize()
    same(out, c.run())


def test_blocks_on_two_streams():
    blocks = [Block(700, 256, 128, 16, 2, seed=s) for s in (0, 100)]
    want = [{n: v.clone() for n, v in b.run().items()} for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [b.run(s) for b, s in zip(blocks, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same(a, b)


class Decode:
    """A decoding step: router -> experts' rows -> gated and down projections on 4-bit weights -> combine."""

    def __init__(self, tokens, hidden, ffn, experts, topk, fmt="int4", group=32):
        self.E, self.K, self.F, self.H, self.fmt, self.group = experts, topk, ffn, hidden, fmt, group
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        self.x, self.logits = randn(21, tokens, hidden), randn(22, tokens, experts)
        codes = lambda r, k: torch.randint(256, (r, k // 2), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
        scales = lambda r, k: (torch.rand((r, k // group), generator=g, device="cuda") * 0.01 + 0.005).bfloat16()  # noqa: E731
        self.w1, self.s1 = codes(experts * 2 * ffn, hidden), scales(experts * 2 * ffn, hidden)
        self.w2, self.s2 = codes(experts * hidden, ffn), scales(experts * hidden, ffn)

    def run(self):
        m, o = te(), {}
        o["experts"], o["weights"] = m.moe_route("softmax", self.logits, self.K)
        o["splits"], o["row_of"], _ = m.moe_sort(o["experts"], self.E)
        o["in"], _, _ = m.moe_dispatch(self.x, o["row_of"])
        o["h"] = m.w4_gemm(o["in"], self.w1, self.fmt, self.s1, activation="silu", m_splits=o["splits"])
        o["out"] = m.w4_gemm(o["h"], self.w2, self.fmt, self.s2, m_splits=o["splits"])
        o["y"] = m.moe_combine(o["out"], o["row_of"], o["weights"])
        return o


@pytest.mark.parametrize("tokens,fmt,group", [(1, "int4", 64), (13, "e2m1", 32), (70, "int4", 128)])
def test_decoding_step(tokens, fmt, group):
    """Relative 2-norms of the whole step in float64: three results rounded to bf16 in a row."""
    d = Decode(tokens, 256, 128, 8, 2, fmt, group)
    o = d.run()
    torch.cuda.synchronize()
    e, w = oracle.route(f(d.logits), 2)
    assert np.array_equal(host(o["experts"]), e)
    w1 = oracle.w4_values(host(d.w1), f(d.s1), fmt).reshape(8, 256, 256)
    w2 = oracle.w4_values(host(d.w2), f(d.s2), fmt).reshape(8, 256, 128)
    x, want = f(d.x), np.zeros((tokens, 256))
    for t, k in np.ndindex(e.shape):
        p = x[t] @ w1[e[t, k]].T
        want[t] += w[t, k] * (w2[e[t, k]] @ (oracle.activation(p[:128], "silu") * p[128:]))
    near(o["y"], want, 3 * 2.0 ** -8)


def test_decoding_step_captured():
    d = Decode(5, 256, 128, 8, 2)
    want = {n: v.clone() for n, v in d.run().items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = d.run()
    for i in range(3):
        for v in out.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        same(out, want)
        d.run()
    x, l = randn(31, 5, 256), randn(32, 5, 8)
    d.x.copy_(x), d.logits.copy_(l)
    g.replay()
    torch.cuda.synchronize()
    same(out, d.run())


def test_rows_past_32_bit_offsets():
    """Tensors of more than 2^31 elements: the last rows, and rows that would lie 2^32 bytes before."""
    T, K, cols = 33000, 2, 34816                                       # 2.3e9 elements, 4.6e9 bytes
    row_of = torch.arange(T * K, dtype=torch.int32, device="cuda").flip(0).view(T, K)
    x = torch.zeros((T, cols), dtype=torch.bfloat16, device="cuda")
    probe = torch.cat([torch.arange(6), torch.arange(T - 6, T)]).cuda()
    x[probe] = randn(41, 12, cols)
    y, _, _ = te().moe_dispatch(x, row_of)
    for t in (0, 3, T - 1):
        for k in range(K):
            assert torch.equal(y[T * K - 1 - t * K - k], x[t])
    w = torch.full((T, K), 0.5, device="cuda")
    back = te().moe_combine(y, row_of, w)                              # half and half of the same row
    assert torch.equal(back[probe], x[probe])
    dw = torch.empty((T, K), device="cuda")
    te().te_moe_combine_backward(x, y, row_of, w, dw, drows=y)         # rows read and written at their own places
    assert torch.equal(y[T * K - 1], x[0] * 0.5) and torch.equal(y[0], x[T - 1] * 0.5)
    want = (f(x[probe]) ** 2).sum(1)
    assert (np.abs(f(dw[probe]) - want[:, None]) <= (cols / 64 + 32) * U * want[:, None]).all()


def test_w4_past_32_bit_offsets():
    """Weights of more than 2^32 bytes: their last columns, against the same columns alone."""
    N, K, group = 530000, 16384, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    w = torch.randint(256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand((N, K // group), generator=g, device="cuda") * 0.01).bfloat16()
    x = randn(51, 3, K)
    whole = te().w4_gemm(x, w, "int4", s)
    for a in (0, N // 2 - 8, N - 48):
        part = te().w4_gemm(x, w[a:a + 48].contiguous(), "int4", s[a:a + 48].contiguous())
        p, size = oracle.w4_gemm(f(x), host(w[a:a + 48]), f(s[a:a + 48]))
        for got in (whole[:, a:a + 48], part):
            assert (np.abs(f(got.contiguous()) - p) <= 2.0 ** -8 * np.abs(p) + (K / 8 + 2 * K / group + 16) * U * size).all()
