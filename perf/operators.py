"""The norm and gated feed-forward operators as they are measured.

Each case is one call of an operator of a LayerNormMLP block with a gated activation:

* ``norm_fwd``   layer norm or RMS norm of a [rows, cols] tensor, with an optional residual add in front (the sum
                 is an output too), to the input's type and / or to a rowwise MXFP8 operand;
* ``norm_bwd``   its backward pass: the input gradient (plus, optionally, the gradient of the skip path) and the
                 gradients of the weight and the bias;
* ``gated_fwd``  act(A Wg' + bg) * (A Wu' + bu) of MXFP8 operands, W = [gate rows; up rows], to bf16 or MXFP8,
                 with the bf16 pre-activations where a backward pass follows; ``groups`` > 0: rows of A dealt
                 to that many experts, each with its own weights;
* ``gated_bwd``  the gradients of both pre-activations from the output gradient's GEMM and the saved
                 pre-activations.

``run`` computes them from elementary torch operations in float32, or with the framework's entry points where
``own`` is true.  MXFP8 outputs are returned as their codes and block scales, typed as the float8 values they are.
"""

import math

import torch

own = False

_FP8 = {"e4m3": (torch.float8_e4m3fn, 8, 448.0, 3, 7), "e5m2": (torch.float8_e5m2, 15, 57344.0, 2, 15)}
_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def _norm(op, rows, cols, dtype="bf16", kind="layer", w="same", residual=False, mx=False, y=True, stats=True):
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "kind": kind, "w": w, "residual": residual,
            "mx": mx, "y": y, "stats": stats}


def _gated(op, m, n, k, act="silu", fmt="e4m3", out="bf16", bias=False, aux=False, groups=0):
    return {"op": op, "m": m, "n": n, "k": k, "act": act, "fmt": fmt, "out": out, "bias": bias, "aux": aux,
            "groups": groups}


def listed():
    return [
        # one token of a decoding step, no statistics kept
        {"name": "norm_fwd_token", **_norm("norm_fwd", 1, 8192, stats=False)},
        # a tensor whose rows are not aligned to anything, in float32
        {"name": "norm_fwd_odd_fp32", **_norm("norm_fwd", 3001, 5003, dtype="fp32")},
        # a long training batch of a wide model: residual add, RMS norm, straight to the next GEMM's operand
        {"name": "norm_fwd_mx_large", **_norm("norm_fwd", 16384, 8192, kind="rms", residual=True, mx=True, y=False)},
        # the decoder layer's tokens and hidden size, training
        {"name": "norm_bwd_decoder", **_norm("norm_bwd", 4096, 1024)},
        # odd sizes in half precision with float32 weights
        {"name": "norm_bwd_odd_fp16", **_norm("norm_bwd", 1021, 2311, dtype="fp16", w="fp32")},
        # the backward pass of the long batch, with the gradient that comes by the skip path
        {"name": "norm_bwd_large", **_norm("norm_bwd", 16384, 8192, kind="rms", residual=True)},
        # one token of a decoding step through a large model's feed-forward block
        {"name": "gated_fwd_token", **_gated("gated_fwd", 1, 14336, 4096)},
        # the decoder layer's tokens, training: bias and saved pre-activations
        {"name": "gated_fwd_decoder", **_gated("gated_fwd", 4096, 4096, 1024, act="gelu", bias=True, aux=True)},
        # a long prompt through a large model's feed-forward block, to the next GEMM's operand
        {"name": "gated_fwd_mx_large", **_gated("gated_fwd", 8192, 14336, 4096, out="e4m3")},
        # ragged tokens over 16 experts
        {"name": "gated_fwd_experts", **_gated("gated_fwd", 8192, 2048, 2048, groups=16)},
        # the decoder layer's backward pass: bound by the pre-activations and their gradients
        {"name": "gated_bwd_decoder", **_gated("gated_bwd", 4096, 4096, 1024, act="gelu")},
        # a large model's backward pass, the output gradient in the wider-range format
        {"name": "gated_bwd_large", **_gated("gated_bwd", 4096, 14336, 4096, fmt="e5m2")},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "gated_fwd", "gated_bwd"))
    if op.startswith("norm"):
        while True:
            rows, cols = _spread(rng, 1, 20000), _spread(rng, 1, 20000)
            if 2000 <= rows * cols <= 60_000_000:
                break
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        kind = rng.choice(("layer", "rms"))
        w = rng.choice(("same", "fp32"))
        residual = rng.random() < 0.5
        if op == "norm_bwd":
            return _norm(op, rows, cols, dtype, kind, w, residual)
        mx = dtype == "bf16" and rng.random() < 0.5
        if mx:
            cols = max(32, cols // 32 * 32)
        return _norm(op, rows, cols, dtype, kind, w, residual, mx, y=not mx or rng.random() < 0.5)
    while True:
        m, n, k = _spread(rng, 1, 8192), _spread(rng, 32, 14336, 32), _spread(rng, 128, 8192, 128)
        if m * n * k <= 8192 * 4096 * 4096 and n * k <= 14336 * 4096:
            break
    act, fmt = rng.choice(("silu", "gelu")), rng.choice(("e4m3", "e5m2"))
    groups = rng.randint(2, 8) if n * k <= 2048 * 2048 and rng.random() < 0.4 else 0
    if op == "gated_bwd":
        return _gated(op, m, n, k, act, fmt, groups=groups)
    out = "bf16" if groups else rng.choice(("bf16", "e4m3"))
    return _gated(op, m, n, k, act, fmt, out, bias=rng.random() < 0.5, aux=rng.random() < 0.5, groups=groups)


# ------------------------------------------------------------------ inputs

def _mx_operand(x, fmt):
    """Rowwise MXFP8 codes and E8M0 scales of x, as a user's program has them before the call."""
    kind, emax, most, _, _ = _FP8[fmt]
    blocks = x.float().view(x.shape[0], -1, 32)
    exp = torch.frexp(blocks.abs().amax(-1, keepdim=True))[1] - 1 - emax
    exp = exp.clamp(-127, 127)
    codes = torch.ldexp(blocks, -exp).clamp(-most, most).to(kind)
    return codes.view(torch.uint8).view(x.shape), (exp[..., 0] + 127).to(torch.uint8)


def _randn(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * sigma).to(dtype)


def _activations(g, rows, cols, dtype):
    """Normal values with a small shift and 1% of the columns 20 times as wide."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    wide = torch.rand(cols, generator=g, device="cuda") < 0.01
    return (x * torch.where(wide, 20.0, 1.0) + 0.125).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    dev = "cuda"
    if c["op"].startswith("norm"):
        dt = _DTYPE[c["dtype"]]
        wt = dt if c["w"] == "same" else torch.float32
        rows, cols = c["rows"], c["cols"]
        s = {"case": c, "x": _activations(g, rows, cols, dt)}
        s["gamma"] = (1 + _randn(g, (cols,), 0.1, torch.float32)).to(wt)
        s["beta"] = _randn(g, (cols,), 0.1, wt) if c["kind"] == "layer" else None
        if c["op"] == "norm_fwd":
            s["residual"] = _randn(g, (rows, cols), 1.0, dt) if c["residual"] else None
            s["sum"] = torch.empty((rows, cols), dtype=dt, device=dev) if c["residual"] else None
            s["y"] = torch.empty((rows, cols), dtype=dt, device=dev) if c["y"] else None
            s["q"] = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if c["mx"] else None
            s["q_scale"] = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev) if c["mx"] else None
            s["mean"] = torch.empty(rows, device=dev) if c["stats"] and c["kind"] == "layer" else None
            s["rstd"] = torch.empty(rows, device=dev) if c["stats"] else None
        else:
            s["dy"] = _randn(g, (rows, cols), 0.01, dt)
            s["dskip"] = _randn(g, (rows, cols), 0.01, dt) if c["residual"] else None
            x = s["x"].double()  # the statistics that the forward pass kept
            mean = x.mean(1) if c["kind"] == "layer" else torch.zeros(rows, device=dev, dtype=torch.float64)
            s["rstd"] = (1 / torch.sqrt((x - mean[:, None]).square().mean(1) + EPS)).float()
            s["mean"] = mean.float() if c["kind"] == "layer" else None
            s["dx"] = torch.empty((rows, cols), dtype=dt, device=dev)
            s["dgamma"] = torch.empty(cols, dtype=wt, device=dev)
            s["dbeta"] = torch.empty(cols, dtype=wt, device=dev) if c["kind"] == "layer" else None
        return s
    m, n, k, groups = c["m"], c["n"], c["k"], c["groups"]
    rows_b = max(groups, 1) * (2 * n if c["op"] == "gated_fwd" else n)
    s = {"case": c, "groups": groups}
    s["a"], s["a_scale"] = _mx_operand(_activations(g, m, k, torch.bfloat16), c["fmt"])
    s["b"], s["b_scale"] = _mx_operand(_randn(g, (rows_b, k), 0.05, torch.bfloat16), "e4m3")
    if groups:
        u = torch.rand(groups, generator=g, device=dev)
        counts = torch.floor(u / u.sum() * m).to(torch.int32)
        counts[-1] += m - counts.sum()
        s["splits"] = counts.to(torch.int32)
        s["most_rows"] = int(counts.max())
    if c["op"] == "gated_fwd":
        s["bias"] = _randn(g, (groups, 2 * n) if groups else (2 * n,), 0.1, torch.bfloat16) if c["bias"] else None
        s["aux"] = torch.empty((m, 2 * n), dtype=torch.bfloat16, device=dev) if c["aux"] else None
        mx = c["out"] != "bf16"
        s["d"] = torch.empty((m, n), dtype=torch.uint8 if mx else torch.bfloat16, device=dev)
        s["d_scale"] = torch.empty((m, n // 32), dtype=torch.uint8, device=dev) if mx else None
    else:
        s["aux"] = _randn(g, (m, 2 * n), 1.0, torch.bfloat16)
        s["d"] = torch.empty((m, 2 * n), dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------------ plain forms

def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)
    return x / (1 + torch.exp(-2 * u))


def _act_grad(x, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s + x * s * (1 - s)
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)
    du = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)
    s = 1 / (1 + torch.exp(-2 * u))
    return s + 2 * x * s * (1 - s) * du


def _values(codes, scales, fmt):
    blocks = codes.view(_FP8[fmt][0]).float().view(codes.shape[0], -1, 32)
    return torch.ldexp(blocks, scales.int()[..., None] - 127).view(codes.shape)


def _typed(codes, scales, fmt):
    return codes.view(_FP8[fmt][0]), scales.view(torch.float8_e8m0fnu)


def _plain_norm_fwd(s):
    c, dt = s["case"], s["x"].dtype
    out = {}
    x = s["x"].float()
    if s["residual"] is not None:
        out["sum"] = (x + s["residual"].float()).to(dt)
        x = out["sum"].float()
    if c["kind"] == "layer":
        mean = x.mean(1, keepdim=True)
        x = x - mean
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    y = y.to(dt)
    if c["y"]:
        out["y"] = y
    if c["mx"]:
        out["q"], out["q_scale"] = _typed(*_mx_operand(y, "e4m3"), "e4m3")
    if c["stats"]:
        out["rstd"] = rstd[:, 0]
        if c["kind"] == "layer":
            out["mean"] = mean[:, 0]
    return out


def _plain_norm_bwd(s):
    c = s["case"]
    x, dy = s["x"].float(), s["dy"].float()
    if c["kind"] == "layer":
        x = x - s["mean"][:, None]
    xh = x * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    if s["dskip"] is not None:
        dx = dx + s["dskip"].float()
    out = {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0).to(s["gamma"].dtype)}
    if s["dbeta"] is not None:
        out["dbeta"] = dy.sum(0).to(s["gamma"].dtype)
    return out


def _plain_product(s):
    """A B' in float32, each row of A with its own expert's B where there are groups."""
    c = s["case"]
    a, b = _values(s["a"], s["a_scale"], c["fmt"]), _values(s["b"], s["b_scale"], "e4m3")
    if not s["groups"]:
        return a @ b.t(), None
    splits = s["splits"].long()
    expert = torch.repeat_interleave(torch.arange(s["groups"], device=a.device), splits, output_size=a.shape[0])
    place = torch.arange(a.shape[0], device=a.device) - (torch.cumsum(splits, 0) - splits)[expert]
    padded = a.new_zeros((s["groups"], s["most_rows"], a.shape[1]))
    padded[expert, place] = a
    b = b.view(s["groups"], -1, a.shape[1]).transpose(1, 2).contiguous()
    return torch.bmm(padded, b)[expert, place], expert


def _plain_gated_fwd(s):
    c, n = s["case"], s["case"]["n"]
    p, expert = _plain_product(s)
    if s["bias"] is not None:
        p = p + (s["bias"].float() if expert is None else s["bias"].float()[expert])
    out = {"aux": p.to(torch.bfloat16)} if c["aux"] else {}
    d = (_act(p[:, :n], c["act"]) * p[:, n:]).to(torch.bfloat16)
    if c["out"] == "bf16":
        out["d"] = d
    else:
        out["d"], out["d_scale"] = _typed(*_mx_operand(d, c["out"]), c["out"])
    return out


def _plain_gated_bwd(s):
    c, n = s["case"], s["case"]["n"]
    dh, _ = _plain_product(s)
    gate, up = s["aux"][:, :n].float(), s["aux"][:, n:].float()
    d = torch.cat((dh * up * _act_grad(gate, c["act"]), dh * _act(gate, c["act"])), 1)
    return {"d": d.to(torch.bfloat16)}


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "gated_fwd": _plain_gated_fwd,
          "gated_bwd": _plain_gated_bwd}


# ------------------------------------------------------------------ the framework's calls

def _own_norm_fwd(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    te.te_norm_forward(c["kind"], s["x"], s["gamma"], s["beta"], EPS, y=s["y"], q=s["q"], q_scale=s["q_scale"],
                       q_fmt="e4m3", residual=s["residual"], sum_out=s["sum"], mean=s["mean"], rstd=s["rstd"])
    out = {}
    if c["residual"]:
        out["sum"] = s["sum"]
    if c["y"]:
        out["y"] = s["y"]
    if c["mx"]:
        out["q"], out["q_scale"] = _typed(s["q"], s["q_scale"], "e4m3")
    if c["stats"]:
        out["rstd"] = s["rstd"]
        if c["kind"] == "layer":
            out["mean"] = s["mean"]
    return out


def _own_norm_bwd(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    if "ws" not in s:  # kept by the program from step to step
        size = te.te_norm_backward_workspace_size(c["rows"], c["cols"])
        s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    te.te_norm_backward(c["kind"], s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"],
                        s["dbeta"], dskip=s["dskip"], workspace=s["ws"])
    out = {"dx": s["dx"], "dgamma": s["dgamma"]}
    if s["dbeta"] is not None:
        out["dbeta"] = s["dbeta"]
    return out


def _own_gated_fwd(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    if s["groups"]:
        te.te_mxfp8_grouped_gated_gemm(s["splits"], s["a"], s["a_scale"], c["fmt"], s["b"], s["b_scale"], "e4m3",
                                       c["n"], s["d"], c["act"], bias=s["bias"], aux=s["aux"])
    else:
        if "ws" not in s:  # kept by the program from step to step
            size = te.te_mxfp8_gated_gemm_workspace_size(c["m"], c["n"], c["k"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        te.te_mxfp8_gated_gemm(s["a"], s["a_scale"], c["fmt"], s["b"], s["b_scale"], "e4m3", s["d"], c["act"],
                               d_scale=s["d_scale"], d_fmt=None if c["out"] == "bf16" else c["out"],
                               bias=s["bias"], aux=s["aux"], workspace=s["ws"])
    out = {"aux": s["aux"]} if c["aux"] else {}
    if c["out"] == "bf16":
        out["d"] = s["d"]
    else:
        out["d"], out["d_scale"] = _typed(s["d"], s["d_scale"], c["out"])
    return out


def _own_gated_bwd(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    if s["groups"]:
        te.te_mxfp8_grouped_dgated_gemm(s["splits"], s["a"], s["a_scale"], c["fmt"], s["b"], s["b_scale"], "e4m3",
                                        c["n"], s["aux"], s["d"], c["act"])
    else:
        if "ws" not in s:  # kept by the program from step to step
            size = te.te_mxfp8_dgated_gemm_workspace_size(c["m"], c["n"], c["k"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        te.te_mxfp8_dgated_gemm(s["a"], s["a_scale"], c["fmt"], s["b"], s["b_scale"], "e4m3", s["aux"], s["d"],
                                c["act"], workspace=s["ws"])
    return {"d": s["d"]}


_OWN = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "gated_fwd": _own_gated_fwd,
        "gated_bwd": _own_gated_bwd}


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"].startswith("norm"):
        e = 4 if c["dtype"] == "fp32" else 2
        we = 4 if c["w"] == "fp32" else e
        rows, cols = c["rows"], c["cols"]
        weights = 2 if c["kind"] == "layer" else 1
        stats = 4 * rows * (2 if c["kind"] == "layer" else 1)
        if c["op"] == "norm_fwd":
            per = e * (1 + 2 * c["residual"] + c["y"]) + (33 / 32 if c["mx"] else 0)
            return {"bytes": rows * cols * per + cols * we * weights + (stats if c["stats"] else 0),
                    "flops": 8 * rows * cols}
        return {"bytes": rows * cols * e * (3 + c["residual"]) + cols * we * (1 + weights) + stats,
                "flops": 14 * rows * cols}
    m, n, k = c["m"], c["n"], c["k"]
    experts = max(c["groups"], 1)
    if c["op"] == "gated_fwd":
        b = (m + experts * 2 * n) * k * 33 / 32 + m * n * (2 if c["out"] == "bf16" else 33 / 32)
        b += 4 * m * n * c["aux"] + experts * 4 * n * c["bias"]
        return {"bytes": b, "flops": 4 * m * n * k}
    return {"bytes": (m + experts * n) * k * 33 / 32 + 8 * m * n, "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits

def _table(fmt):
    """The 256 values of an FP8 format from its definition: sign, exponent and mantissa fields."""
    _, _, most, man, bias = _FP8[fmt]
    values = []
    for code in range(256):
        e, f = (code >> man) & ((1 << (7 - man)) - 1), code & ((1 << man) - 1)
        v = math.ldexp(f, 1 - bias - man) if e == 0 else math.ldexp((1 << man) + f, e - bias - man)
        values.append((-v if code & 128 else v) if v <= most else math.nan)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _exact_values(codes, scales, fmt):
    v = _table(fmt)[codes.long()]
    power = torch.pow(2.0, scales.double() - 127)
    return v * power.repeat_interleave(32, dim=1)


def _exact_mx(y, fmt):
    """Codes and scales (as values) of the rowwise MXFP8 operand of the bf16 values y, in 64 bits."""
    _, emax, most, man, bias = _FP8[fmt]
    blocks = y.view(y.shape[0], -1, 32)
    amax = blocks.abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 2.0 ** -140)))) - emax
    scale = torch.pow(2.0, e.clamp(min=-127.0))
    v = blocks / scale[..., None]
    # the quantum of each value: 2^(its exponent - mantissa bits), not below the subnormals' one
    at = torch.where(v == 0, torch.full_like(v, 2.0 ** -60), v.abs())
    quantum = torch.pow(2.0, torch.floor(torch.log2(at)).clamp(min=1 - bias) - man)
    v = (torch.round(v / quantum) * quantum).clamp(-most, most)
    return v.view(y.shape), scale


def _exact_act(x, act, grad=False):
    if act == "silu":
        s = torch.sigmoid(x)
        return s * (1 + x * (1 - s)) if grad else x * s
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (x + 0.044715 * x ** 3))
    if not grad:
        return 0.5 * x * (1 + t)
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 3 * 0.044715 * x ** 2)


def _exact_norm(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"].double()
    out = {}
    if c["op"] == "norm_fwd":
        if c["residual"]:
            out["sum"] = x + s["residual"].double()
            x = out["sum"].to(dt).double()
        mean = x.sum(1) / c["cols"] if c["kind"] == "layer" else torch.zeros_like(x[:, 0])
        x = x - mean[:, None]
        rstd = 1 / torch.sqrt((x * x).sum(1) / c["cols"] + EPS)
        y = x * rstd[:, None] * s["gamma"].double()
        if s["beta"] is not None:
            y = y + s["beta"].double()
        if c["y"]:
            out["y"] = y
        if c["mx"]:
            out["q"], out["q_scale"] = _exact_mx(y.to(torch.bfloat16).double(), "e4m3")
        if c["stats"]:
            out["rstd"] = rstd
            if c["kind"] == "layer":
                out["mean"] = mean
        return out
    dy, gamma, rstd = s["dy"].double(), s["gamma"].double(), s["rstd"].double()[:, None]
    xh = (x - s["mean"].double()[:, None] if c["kind"] == "layer" else x) * rstd
    g = dy * gamma
    n = c["cols"]
    dx = rstd / n * (n * g - xh * (g * xh).sum(1)[:, None] - (g.sum(1)[:, None] if c["kind"] == "layer" else 0))
    if s["dskip"] is not None:
        dx = dx + s["dskip"].double()
    out = {"dx": dx, "dgamma": (dy * xh).sum(0)}
    if s["dbeta"] is not None:
        out["dbeta"] = dy.sum(0)
    return out


def _exact_gated(s):
    c, n = s["case"], s["case"]["n"]
    a = _exact_values(s["a"], s["a_scale"], c["fmt"])
    b = _exact_values(s["b"], s["b_scale"], "e4m3")
    if s["groups"]:
        parts, per = [], b.shape[0] // s["groups"]
        for e, rows in enumerate(torch.split(a, s["splits"].tolist())):
            p = torch.matmul(rows, b[e * per:(e + 1) * per].transpose(0, 1).contiguous())
            if c["op"] == "gated_fwd" and s["bias"] is not None:
                p = p + s["bias"][e].double()
            parts.append(p)
        p = torch.cat(parts)
    else:
        p = torch.matmul(a, b.transpose(0, 1).contiguous())
        if c["op"] == "gated_fwd" and s["bias"] is not None:
            p = p + s["bias"].double()
    if c["op"] == "gated_bwd":
        gate, up = s["aux"].double().split(n, dim=1)
        return {"d": torch.cat((p * up * _exact_act(gate, c["act"], grad=True), p * _exact_act(gate, c["act"])), 1)}
    out = {"aux": p} if c["aux"] else {}
    d = _exact_act(p[:, :n], c["act"]) * p[:, n:]
    if c["out"] == "bf16":
        out["d"] = d
    else:
        out["d"], out["d_scale"] = _exact_mx(d.to(torch.bfloat16).double(), c["out"])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_gated(s)
