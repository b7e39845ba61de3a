"""The operators around and beside the grouped GEMM of a mixture-of-experts block, as they are measured.

Each case is one call of an operator (the sort and the dispatch are one: a program makes both calls in a row):

* ``route_fwd``    the router: each token's ``topk`` experts and their weights from its logits;
* ``route_bwd``    the logits' gradient from the weights' one;
* ``dispatch_fwd`` the tokens sorted by expert: the rows' numbers, the experts' row counts, and the rows themselves,
                   in the tokens' type or as the grouped GEMM's MXFP8 operand;
* ``dispatch_bwd`` its gradient: each token's rows added up;
* ``combine_fwd``  each token's rows, by now the experts' outputs, added up with the router's weights;
* ``combine_bwd``  the gradients of the rows and of the weights;
* ``w4``           X W' of few rows with 4-bit weights and group scales (dense, or ``groups`` experts with their own
                   weights), plain or gated: act(X Wg') * (X Wu') with W = [gate rows; up rows].

``run`` computes them from elementary torch operations in float32, or with the framework's entry points where
``own`` is true.  MXFP8 outputs are returned as their codes and block scales, typed as the float8 values they are.
"""

import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e8m0": 1}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of the format's codes


# ------------------------------------------------------------------ the cases

def _route(op, tokens, experts, topk, score="softmax", normalize=True, scale=1.0, bias=False, dtype="fp32",
           masked=False):
    return {"op": op, "tokens": tokens, "experts": experts, "topk": topk, "score": score, "normalize": normalize,
            "scale": scale, "bias": bias, "dtype": dtype, "masked": masked}


def _rows(op, tokens, experts, topk, cols, dtype="bf16", mx=False, masked=False):
    return {"op": op, "tokens": tokens, "experts": experts, "topk": topk, "cols": cols, "dtype": dtype, "mx": mx,
            "masked": masked}


def _w4(m, n, k, group, fmt="int4", scales="bf16", zeros=False, dtype="bf16", act="none", bias=False, groups=0):
    return {"op": "w4", "m": m, "n": n, "k": k, "group": group, "fmt": fmt, "scales": scales, "zeros": zeros,
            "dtype": dtype, "act": act, "bias": bias, "groups": groups}


def listed():
    return [
        # one token of a decoding step
        {"name": "route_token", **_route("route_fwd", 1, 32, 2, dtype="bf16")},
        # a long training batch over many experts, selected with a balancing bias
        {"name": "route_large", **_route("route_fwd", 16384, 256, 8, score="sigmoid", scale=2.5, bias=True)},
        # its gradient for a router whose weights are shares of all the experts, odd sizes
        {"name": "route_bwd_odd", **_route("route_bwd", 5003, 60, 4, normalize=False, dtype="bf16")},
        # one token of a decoding step to its experts
        {"name": "dispatch_token", **_rows("dispatch_fwd", 1, 32, 2, 4096)},
        # a long training batch over many experts, straight to the grouped GEMM's operand
        {"name": "dispatch_mx_large", **_rows("dispatch_fwd", 16384, 256, 8, 4096, mx=True)},
        # the gradient of the benchmark's 16384 routed rows, two experts a token
        {"name": "dispatch_bwd_benchmark", **_rows("dispatch_bwd", 8192, 32, 2, 4096)},
        # odd sizes in half precision, with padding tokens
        {"name": "combine_odd_fp16", **_rows("combine_fwd", 3001, 60, 6, 2311, dtype="fp16", masked=True)},
        # the backward pass of a long batch over many experts
        {"name": "combine_bwd_large", **_rows("combine_bwd", 8192, 256, 8, 4096)},
        # one token of a decoding step through a large model's gated projections
        {"name": "w4_token", **_w4(1, 14336, 4096, 128, act="silu")},
        # batched decoding through its down projection, weights in the 4-bit MX format
        {"name": "w4_batch", **_w4(32, 4096, 14336, 32, fmt="e2m1", scales="e8m0")},
        # odd sizes: small groups with zero points, in half precision
        {"name": "w4_odd_fp16", **_w4(5, 1001, 2080, 32, scales="fp16", zeros=True, dtype="fp16", bias=True)},
        # a decoding batch's rows over the benchmark's experts
        {"name": "w4_experts", **_w4(64, 1536, 4096, 128, groups=32)},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(("route_fwd", "route_bwd", "dispatch_fwd", "dispatch_bwd", "combine_fwd", "combine_bwd", "w4", "w4",
                     "w4"))
    if op.startswith("route"):
        while True:
            tokens, experts = _spread(rng, 1, 32768), _spread(rng, 2, 1024)
            if tokens * experts <= 16384 * 256:
                break
        score = rng.choice(("softmax", "sigmoid"))
        return _route(op, tokens, experts, min(experts, rng.randint(1, 10)), score, rng.random() < 0.6,
                      rng.choice((1.0, 2.5)), op == "route_fwd" and rng.random() < 0.4,
                      rng.choice(("fp32", "fp32", "bf16", "fp16")), rng.random() < 0.3)
    if op != "w4":
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        mx = dtype == "bf16" and op in ("dispatch_fwd", "combine_bwd") and rng.random() < 0.5
        while True:
            tokens, experts, cols = _spread(rng, 1, 16384), _spread(rng, 2, 512), _spread(rng, 1, 9000)
            topk = min(experts, rng.randint(1, 8))
            if mx:
                cols = max(32, cols // 32 * 32)
            if tokens * topk * cols <= 8192 * 8 * 4096 * 2 // _SIZE[dtype]:
                break
        return _rows(op, tokens, experts, topk, cols, dtype, mx, rng.random() < 0.3)
    group = rng.choice((32, 32, 64, 128, 128, 256))
    groups = rng.randint(2, 64) if rng.random() < 0.4 else 0
    act = rng.choice(("none", "none", "silu", "gelu"))
    while True:
        m, n, k = _spread(rng, 1, 256), _spread(rng, 1, 28672), _spread(rng, group, 16384, group)
        weights = max(groups, 1) * n * k * (1 if act == "none" else 2)
        if 4096 <= weights <= 28672 * 4096 and m * weights <= 32 * 4096 * 14336:
            break
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    fmt = rng.choice(("int4", "int4", "e2m1"))
    scales = rng.choice((dtype, "fp32") if fmt == "int4" else ("e8m0", "e8m0", dtype, "fp32"))
    return _w4(m, n, k, group, fmt, scales, fmt == "int4" and rng.random() < 0.5, dtype, act, rng.random() < 0.3, groups)


# ------------------------------------------------------------------ inputs

def _randn(g, shape, sigma, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * sigma).to(dtype)


def _activations(g, rows, cols, dtype):
    """Normal values with a small shift and 1% of the columns 20 times as wide."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    wide = torch.rand(cols, generator=g, device="cuda") < 0.01
    return (x * torch.where(wide, 20.0, 1.0) + 0.125).to(dtype)


def _logits(g, c):
    """Router logits: some experts are liked by every token; masked: a few logits and a few whole tokens are left out."""
    t, e = c["tokens"], c["experts"]
    x = _randn(g, (t, e), 1.0) + _randn(g, (e,), 0.5)
    if c["masked"]:
        out = (torch.rand((t, e), generator=g, device="cuda") < 0.03) | (torch.rand((t, 1), generator=g, device="cuda") < 0.05)
        x = torch.where(out, -math.inf, x)
    return x


def _chosen(logits, topk):
    """Experts int32 [tokens, topk] in falling order of the logits, -1 where only masked ones are left."""
    values, experts = torch.topk(logits, topk, dim=1)
    return torch.where(values > -math.inf, experts, -1).to(torch.int32)


def _maps(experts, num_experts):
    """Of a stable sort of the slots by expert: each slot's row (-1: none) and the rows in all."""
    flat = experts.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, num_experts, flat), stable=True)[1]
    row_of = torch.empty_like(flat)
    row_of[order] = torch.arange(flat.numel(), device=flat.device)
    return torch.where(flat < 0, -1, row_of).to(torch.int32).view(experts.shape)


def _w4_weights(g, c, rows):
    """Codes, two a byte (even k in the low half), scales and zero points of normal weights."""
    k, group = c["k"], c["group"]
    codes, scales, zeros = [], [], []
    for part in torch.split(torch.arange(rows), max(1, (1 << 26) // k)):  # in pieces: the float32 weights are large
        w = _randn(g, (len(part), k // group, group), 0.02)
        if c["fmt"] == "e2m1":
            amax = w.abs().amax(-1)
            s = torch.ldexp(torch.ones_like(amax), torch.frexp(amax)[1] - 3)
            if c["scales"] != "e8m0":
                s = (amax / 6).to(_DTYPE[c["scales"]])
            grid = torch.tensor(_E2M1, device="cuda")
            q = torch.bucketize((w / s.float()[..., None]).abs(), (grid[1:] + grid[:-1]) / 2)
            q = q + 8 * (w < 0)
            if c["scales"] == "e8m0":
                s = (torch.frexp(s)[1] + 126).to(torch.uint8)
        elif c["zeros"]:
            low, high = w.amin(-1), w.amax(-1)
            s = ((high - low) / 15).to(_DTYPE[c["scales"]])
            z = torch.round(-low / s.float())
            q = torch.round(w / s.float()[..., None] + z[..., None]).clamp(0, 15)
            zeros.append(z.to(torch.uint8))
        else:
            s = (w.abs().amax(-1) / 7).to(_DTYPE[c["scales"]])
            q = (torch.round(w / s.float()[..., None]) + 8).clamp(0, 15)
        q = q.view(len(part), k // 2, 2).to(torch.uint8)
        codes.append(q[..., 0] | q[..., 1] << 4)
        scales.append(s)
    return torch.cat(codes), torch.cat(scales), torch.cat(zeros) if zeros else None


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "w4":
        dt, m, n = _DTYPE[c["dtype"]], c["m"], c["n"]
        experts = max(c["groups"], 1)
        rows = n if c["act"] == "none" else 2 * n
        s["x"] = _activations(g, m, c["k"], dt)
        s["w"], s["scale"], s["zero"] = _w4_weights(g, c, experts * rows)
        s["bias"] = _randn(g, (experts, rows) if c["groups"] else (rows,), 0.1, dt) if c["bias"] else None
        if c["groups"]:  # a routed batch: each row's expert by chance, the rows in order
            to = torch.randint(experts, (m,), generator=g, device="cuda")
            s["splits"] = torch.zeros(experts, dtype=torch.int32, device="cuda").index_add_(
                0, to, torch.ones(m, dtype=torch.int32, device="cuda"))
            s["most_rows"] = int(s["splits"].max())
        s["d"] = torch.empty((m, n), dtype=dt, device="cuda")
        return s
    t, e, k = c["tokens"], c["experts"], c["topk"]
    logits = _logits(g, c)
    if c["op"].startswith("route"):
        s["logits"] = logits.to(_DTYPE[c["dtype"]])
        if c["op"] == "route_fwd":
            s["bias"] = _randn(g, (e,), 0.1) if c["bias"] else None
            s["experts"] = torch.empty((t, k), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((t, k), device="cuda")
        else:
            s["experts"] = _chosen(s["logits"].float(), k)
            s["dweights"] = _randn(g, (t, k), 0.1)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    dt, cols = _DTYPE[c["dtype"]], c["cols"]
    s["experts"] = _chosen(logits, k)
    if c["op"] == "dispatch_fwd":
        s["x"] = _activations(g, t, cols, dt)
        s["row_of"] = torch.empty((t, k), dtype=torch.int32, device="cuda")
        s["slot_of"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
        s["splits"] = torch.empty(e, dtype=torch.int32, device="cuda")
    else:
        s["row_of"] = _maps(s["experts"], e)
        if c["op"] == "dispatch_bwd":
            s["drows"] = _randn(g, (t * k, cols), 0.01, dt)
        else:
            s["rows"] = _randn(g, (t * k, cols), 1.0, dt)
            s["weights"] = torch.softmax(_randn(g, (t, k), 1.0), 1)
        if c["op"] == "combine_bwd":
            s["dy"] = _randn(g, (t, cols), 0.01, dt)
            s["dweights"] = torch.empty((t, k), device="cuda")
        else:
            s["y"] = torch.empty((t, cols), dtype=dt, device="cuda")
    if c["op"] in ("dispatch_fwd", "combine_bwd"):
        # rows behind the last are not written: zeros from the start
        if c["mx"]:
            s["q"] = torch.zeros((t * k, cols), dtype=torch.uint8, device="cuda")
            s["q_scale"] = torch.zeros((t * k, cols // 32), dtype=torch.uint8, device="cuda")
        else:
            s["out"] = torch.zeros((t * k, cols), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _mx_operand(x, fmt):
    """Rowwise MXFP8 codes and E8M0 scales of x."""
    kind, emax, most = {"e4m3": (torch.float8_e4m3fn, 8, 448.0), "e5m2": (torch.float8_e5m2, 15, 57344.0)}[fmt]
    blocks = x.float().view(x.shape[0], -1, 32)
    exp = (torch.frexp(blocks.abs().amax(-1, keepdim=True))[1] - 1 - emax).clamp(-127, 127)
    codes = torch.ldexp(blocks, -exp).clamp(-most, most).to(kind)
    return codes.view(torch.uint8).view(x.shape), (exp[..., 0] + 127).to(torch.uint8)


def _typed(codes, scales, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2), scales.view(torch.float8_e8m0fnu)


def _scores(x, live, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = torch.where(live.any(1, keepdim=True), x.amax(1, keepdim=True), 0)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, 1)


def _plain_route_fwd(s):
    c = s["case"]
    x = s["logits"].float()
    live = x > -math.inf
    key = x  # the scores rise with the logits
    if s["bias"] is not None:  # two of these may lie next to each other: in 64 bits
        key = torch.where(live, _scores(x.double(), live, c["score"]) + s["bias"].double(), -math.inf)
    experts = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :c["topk"]]
    live = torch.gather(live, 1, experts)
    w = torch.where(live, torch.gather(_scores(x, x > -math.inf, c["score"]), 1, experts), 0)
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1)
    return {"experts": torch.where(live, experts, -1).to(torch.int32), "weights": w * c["scale"]}


def _plain_route_bwd(s):
    c = s["case"]
    x = s["logits"].float()
    live = x > -math.inf
    p = _scores(x, live, c["score"])
    slot = s["experts"] >= 0
    at = torch.where(slot, s["experts"], 0).long()
    w = torch.where(slot, torch.gather(p, 1, at), 0)
    ds = torch.where(slot, s["dweights"] * c["scale"], 0)
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1)
        ds = (ds - (ds * w).sum(1, keepdim=True) / total) / total
        ds = torch.where(slot, ds, 0)
    ds = torch.zeros_like(p).scatter_add_(1, at, ds)
    if c["score"] == "sigmoid":
        d = ds * p * (1 - p)
    else:
        d = p * (ds - (ds * p).sum(1, keepdim=True))
    return {"dlogits": d.to(s["logits"].dtype)}


def _scattered(rows, row_of):
    """rows[slot] in the place of each slot's row, zeros behind the last."""
    out = rows.new_zeros(rows.shape)
    flat = row_of.reshape(-1).long()
    keep = torch.sort((flat < 0).to(torch.int8), stable=True)[1]  # slots that have a row first
    at = flat[keep]
    n = rows.shape[0]
    at = torch.where(at < 0, torch.arange(n, device=rows.device), at)  # the others' places: behind the last row
    gone = (flat[keep] < 0).view(-1, *([1] * (rows.dim() - 1)))
    out[at] = torch.where(gone, torch.zeros((), dtype=rows.dtype, device=rows.device), rows[keep])
    return out


def _plain_dispatch_fwd(s):
    c, k = s["case"], s["case"]["topk"]
    flat = s["experts"].reshape(-1).long()
    n, e = flat.numel(), c["experts"]
    key = torch.where(flat < 0, e, flat)
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(e + 1, dtype=torch.int32, device=flat.device)
    counts.index_add_(0, key, torch.ones(n, dtype=torch.int32, device=flat.device))
    row_of = torch.empty_like(flat)
    row_of[order] = torch.arange(n, device=flat.device)
    row_of = torch.where(flat < 0, -1, row_of)
    there = torch.arange(n, device=flat.device) < n - counts[e]
    out = {"row_of": row_of.to(torch.int32).view(s["experts"].shape), "splits": counts[:e],
           "slot_of": torch.where(there, order, -1).to(torch.int32)}
    token = torch.div(order, k, rounding_mode="floor")
    if c["mx"]:
        q, scale = _mx_operand(s["x"], "e4m3")
        out["q"], out["q_scale"] = _typed(torch.where(there[:, None], q[token], 0),
                                          torch.where(there[:, None], scale[token], 0), "e4m3")
    else:
        out["y"] = torch.where(there[:, None], s["x"][token], 0)
    return out


def _gathered(rows, row_of):
    """[tokens, topk, cols]: each slot's row in float32, zeros where it has none."""
    at = torch.where(row_of < 0, 0, row_of).long()
    return torch.where((row_of < 0)[..., None], 0, rows[at].float())


def _plain_dispatch_bwd(s):
    return {"dx": _gathered(s["drows"], s["row_of"]).sum(1).to(s["drows"].dtype)}


def _plain_combine_fwd(s):
    y = (_gathered(s["rows"], s["row_of"]) * s["weights"][..., None]).sum(1)
    return {"y": y.to(s["rows"].dtype)}


def _plain_combine_bwd(s):
    c = s["case"]
    dy = s["dy"].float()
    rows = _gathered(s["rows"], s["row_of"])
    out = {"dweights": (rows * dy[:, None, :]).sum(2)}
    del rows
    d = (s["weights"][..., None] * dy[:, None, :]).to(s["rows"].dtype)
    d = _scattered(d.view(-1, c["cols"]), s["row_of"])
    if c["mx"]:
        q, scale = _mx_operand(d, "e5m2")
        there = (torch.arange(d.shape[0], device=d.device) < (s["row_of"] >= 0).sum())[:, None]
        out["q"], out["q_scale"] = _typed(q, torch.where(there, scale, 0), "e5m2")
    else:
        out["drows"] = d
    return out


def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)
    return x / (1 + torch.exp(-2 * u))


def _plain_w4(s):
    c, n = s["case"], s["case"]["n"]
    w = torch.stack((s["w"] & 15, s["w"] >> 4), -1).view(s["w"].shape[0], -1, c["group"])
    if c["fmt"] == "e2m1":
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=w.device)
        w = table[w.int()]
    else:
        w = w.float() - (8.0 if s["zero"] is None else s["zero"].float()[..., None])
    scale = torch.exp2(s["scale"].float() - 127) if c["scales"] == "e8m0" else s["scale"].float()
    w = (w * scale[..., None]).view(-1, c["k"])
    x = s["x"].float()
    expert = None
    if not c["groups"]:
        p = x @ w.t()
    else:
        splits = s["splits"].long()
        expert = torch.repeat_interleave(torch.arange(c["groups"], device=w.device), splits, output_size=c["m"])
        place = torch.arange(c["m"], device=w.device) - (torch.cumsum(splits, 0) - splits)[expert]
        padded = x.new_zeros((c["groups"], s["most_rows"], c["k"]))
        padded[expert, place] = x
        p = torch.bmm(padded, w.view(c["groups"], -1, c["k"]).transpose(1, 2).contiguous())[expert, place]
    if s["bias"] is not None:
        p = p + (s["bias"].float() if expert is None else s["bias"].float()[expert])
    if c["act"] != "none":
        p = _act(p[:, :n], c["act"]) * p[:, n:]
    return {"d": p.to(s["x"].dtype)}


_PLAIN = {"route_fwd": _plain_route_fwd, "route_bwd": _plain_route_bwd, "dispatch_fwd": _plain_dispatch_fwd,
          "dispatch_bwd": _plain_dispatch_bwd, "combine_fwd": _plain_combine_fwd, "combine_bwd": _plain_combine_bwd,
          "w4": _plain_w4}


# ------------------------------------------------------------------ the framework's calls

def _own_route_fwd(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    te.te_moe_route(c["score"], s["logits"], s["experts"], s["weights"], bias=s["bias"], normalize=c["normalize"],
                    scale=c["scale"])
    return {"experts": s["experts"], "weights": s["weights"]}


def _own_route_bwd(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    te.te_moe_route_backward(c["score"], s["logits"], s["experts"], s["dweights"], s["dlogits"],
                             normalize=c["normalize"], scale=c["scale"])
    return {"dlogits": s["dlogits"]}


def _own_dispatch_fwd(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    if "ws" not in s:  # kept by the program from step to step
        size = te.te_moe_sort_workspace_size(s["experts"].numel(), c["experts"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    te.te_moe_sort(s["experts"], s["splits"], s["row_of"], s["slot_of"], workspace=s["ws"])
    out = {"row_of": s["row_of"], "slot_of": s["slot_of"], "splits": s["splits"]}
    if c["mx"]:
        te.te_moe_dispatch(s["x"], s["row_of"], q=s["q"], q_scale=s["q_scale"], q_fmt="e4m3")
        out["q"], out["q_scale"] = _typed(s["q"], s["q_scale"], "e4m3")
    else:
        te.te_moe_dispatch(s["x"], s["row_of"], y=s["out"])
        out["y"] = s["out"]
    return out


def _own_dispatch_bwd(s):
    import mxfp8_mixed_precision_amd as te
    te.te_moe_combine(s["drows"], s["row_of"], s["y"])
    return {"dx": s["y"]}


def _own_combine_fwd(s):
    import mxfp8_mixed_precision_amd as te
    te.te_moe_combine(s["rows"], s["row_of"], s["y"], weights=s["weights"])
    return {"y": s["y"]}


def _own_combine_bwd(s):
    import mxfp8_mixed_precision_amd as te
    out = {"dweights": s["dweights"]}
    if s["case"]["mx"]:
        te.te_moe_combine_backward(s["dy"], s["rows"], s["row_of"], s["weights"], s["dweights"], q=s["q"],
                                   q_scale=s["q_scale"], q_fmt="e5m2")
        out["q"], out["q_scale"] = _typed(s["q"], s["q_scale"], "e5m2")
    else:
        te.te_moe_combine_backward(s["dy"], s["rows"], s["row_of"], s["weights"], s["dweights"], drows=s["out"])
        out["drows"] = s["out"]
    return out


def _own_w4(s):
    import mxfp8_mixed_precision_amd as te
    c = s["case"]
    more = {"zero": s["zero"], "bias": s["bias"]}
    if c["groups"] and c["act"] != "none":
        te.te_w4_grouped_gated_gemm(s["splits"], s["x"], s["w"], c["fmt"], s["scale"], c["n"], s["d"], c["act"], **more)
    elif c["groups"]:
        te.te_w4_grouped_gemm(s["splits"], s["x"], s["w"], c["fmt"], s["scale"], c["n"], s["d"], **more)
    elif c["act"] != "none":
        te.te_w4_gated_gemm(s["x"], s["w"], c["fmt"], s["scale"], s["d"], c["act"], **more)
    else:
        te.te_w4_gemm(s["x"], s["w"], c["fmt"], s["scale"], s["d"], **more)
    return {"d": s["d"]}


_OWN = {"route_fwd": _own_route_fwd, "route_bwd": _own_route_bwd, "dispatch_fwd": _own_dispatch_fwd,
        "dispatch_bwd": _own_dispatch_bwd, "combine_fwd": _own_combine_fwd, "combine_bwd": _own_combine_bwd,
        "w4": _own_w4}


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "w4":
        m, n, k, e = c["m"], c["n"], c["k"], max(c["groups"], 1)
        rows = n if c["act"] == "none" else 2 * n
        used = e * (1 - (1 - 1 / e) ** m) if e > 1 else 1  # experts that have rows
        weights = rows * k / 2 + rows * (k // c["group"]) * (_SIZE[c["scales"]] + c["zeros"]) + 2 * rows * c["bias"]
        return {"bytes": used * weights + 2 * m * (k + n) + (4 * e if c["groups"] else 0), "flops": 2 * m * rows * k}
    t, e, k, size = c["tokens"], c["experts"], c["topk"], _SIZE[c["dtype"]]
    if c["op"] == "route_fwd":
        return {"bytes": t * e * size + 8 * t * k + 4 * e * c["bias"], "flops": 8 * t * e + 4 * t * k}
    if c["op"] == "route_bwd":
        read = k if c["normalize"] or c["score"] == "sigmoid" else e  # the chosen experts' logits, or all
        return {"bytes": t * (e + read) * size + 8 * t * k, "flops": 8 * t * e}
    cols = c["cols"]
    if c["op"] == "dispatch_fwd":
        out = cols * 33 / 32 if c["mx"] else cols * size
        return {"bytes": 12 * t * k + 4 * e + t * cols * size + t * k * out, "flops": t * cols * 2 * (1 + c["mx"])}
    if c["op"] == "combine_bwd":
        out = cols * 33 / 32 if c["mx"] else cols * size
        return {"bytes": 12 * t * k + t * cols * size * (1 + k) + t * k * out, "flops": 3 * t * k * cols}
    return {"bytes": 8 * t * k + t * cols * size * (1 + k), "flops": 2 * t * k * cols}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_mx(y, fmt):
    """Codes and scales (as values) of the rowwise MXFP8 operand of the bf16 values y, in 64 bits."""
    emax, most, man, bias = {"e4m3": (8, 448.0, 3, 7), "e5m2": (15, 57344.0, 2, 15)}[fmt]
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


def _exact_weights(x, experts, c):
    """The weights of given experts, differentiable: softmax over all, or sigmoid, then shares of the chosen."""
    there = experts >= 0
    at = experts.clamp(min=0).long()
    if c["score"] == "sigmoid":
        w = torch.sigmoid(x).gather(1, at)
    else:
        none = torch.isinf(x).all(1, keepdim=True)
        w = torch.softmax(x.masked_fill(none, 0.0), 1).gather(1, at)
    w = w.masked_fill(~there, 0.0)
    if c["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / total.masked_fill(total == 0, 1.0)
    return c["scale"] * w


def _exact_route(s):
    c, x = s["case"], s["logits"].double()
    if c["op"] == "route_bwd":
        x.requires_grad_(True)
        _exact_weights(x, s["experts"], c).backward(s["dweights"].double())
        return {"dlogits": x.grad.masked_fill(torch.isinf(s["logits"]), 0.0)}
    key = x.clone()
    if s["bias"] is not None:
        none = torch.isinf(x).all(1, keepdim=True)
        key = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x.masked_fill(none, 0.0), 1)
        key = (key + s["bias"].double()).masked_fill(torch.isinf(x), -math.inf)
    found = []
    for _ in range(c["topk"]):  # the largest key that is left, the first of equal ones
        best = key.amax(1, keepdim=True)
        first = (key == best).to(torch.int8).argmax(1, keepdim=True)
        found.append(torch.where(torch.isinf(best), -1, first))
        key = key.scatter(1, first, -math.inf)
    experts = torch.cat(found, 1)
    return {"experts": experts.to(torch.int32), "weights": _exact_weights(x, experts, c)}


def _exact_rows(s):
    c, k = s["case"], s["case"]["topk"]
    flat = s["experts"].reshape(-1)
    # a slot's row: the slots of smaller experts, and the earlier ones of its own
    slots = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(c["experts"])])
    rows, n = slots.numel(), flat.numel()
    row_of = torch.full((n,), -1, dtype=torch.int32, device=flat.device)
    row_of[slots] = torch.arange(rows, dtype=torch.int32, device=flat.device)
    if c["op"] == "dispatch_fwd":
        slot_of = torch.full((n,), -1, dtype=torch.int32, device=flat.device)
        slot_of[:rows] = slots.to(torch.int32)
        splits = torch.stack([(flat == e).sum() for e in range(c["experts"])]).to(torch.int32)
        out = {"row_of": row_of.view(s["experts"].shape), "slot_of": slot_of, "splits": splits}
        if not c["mx"]:
            y = s["x"].new_zeros((n, c["cols"]))
            y[:rows] = s["x"][slots // k]
            return {**out, "y": y}
        v, scale = _exact_mx(s["x"].double(), "e4m3")
        out["q"] = torch.zeros((n, c["cols"]), dtype=torch.float32, device=flat.device)
        out["q"][:rows] = v.float()[slots // k]
        out["q_scale"] = torch.full((n, c["cols"] // 32), 2.0 ** -127, dtype=torch.float64, device=flat.device)
        out["q_scale"][:rows] = scale[slots // k]
        return out
    if c["op"] == "combine_bwd":
        dy, w = s["dy"].double(), s["weights"].double().view(-1)
        dweights = torch.zeros(n, dtype=torch.float64, device=flat.device)
        for part in torch.split(torch.arange(rows, device=flat.device), 1 << 14):
            dweights[slots[part]] = (s["rows"][part].double() * dy[slots[part] // k]).sum(1)
        out = {"dweights": dweights.view(s["experts"].shape)}
        d = torch.zeros((n, c["cols"]), dtype=torch.float64, device=flat.device)
        d[:rows] = w[slots, None] * dy[slots // k]
        if not c["mx"]:
            return {**out, "drows": d}
        out["q"], out["q_scale"] = _exact_mx(d.to(torch.bfloat16).double(), "e5m2")
        out["q_scale"][rows:] = 2.0 ** -127
        return out
    y = torch.zeros((c["tokens"], c["cols"]), dtype=torch.float64, device=flat.device)
    rows_in = s["drows"] if c["op"] == "dispatch_bwd" else s["rows"]
    for j in range(k):
        at = row_of.view(-1, k)[:, j].long()
        there = at >= 0
        w = 1.0 if c["op"] == "dispatch_bwd" else s["weights"][there, j].double()[:, None]
        y[there] += w * rows_in[at[there]].double()
    return {"dx" if c["op"] == "dispatch_bwd" else "y": y}


def _exact_w4(s):
    c, n = s["case"], s["case"]["n"]
    experts = max(c["groups"], 1)
    splits = s["splits"].tolist() if c["groups"] else [c["m"]]
    per = s["w"].shape[0] // experts
    parts, at = [], 0
    for e, m in enumerate(splits):
        if m == 0:
            continue
        rows = slice(e * per, (e + 1) * per)
        codes = s["w"][rows].long()
        w = torch.empty((per, c["k"]), dtype=torch.float64, device=codes.device)
        w[:, 0::2], w[:, 1::2] = (codes % 16).double(), (codes // 16).double()
        if c["fmt"] == "e2m1":  # sign, 2 bits of exponent (bias 1), 1 of mantissa
            q = w.long()
            e2, man = (q // 2) % 4, q % 2
            w = torch.where(e2 == 0, 0.5 * man, (1 + 0.5 * man) * torch.pow(2.0, e2.double() - 1)) * (1 - 2 * (q // 8))
        else:
            zero = 8.0 if s["zero"] is None else s["zero"][rows].double().repeat_interleave(c["group"], 1)
            w = w - zero
        scale = s["scale"][rows].double()
        scale = torch.pow(2.0, scale - 127) if c["scales"] == "e8m0" else scale
        w = w * scale.repeat_interleave(c["group"], 1)
        p = torch.matmul(s["x"][at:at + m].double(), w.transpose(0, 1).contiguous())
        at += m
        if s["bias"] is not None:
            p = p + (s["bias"][e] if c["groups"] else s["bias"]).double()
        parts.append(p)
    p = torch.cat(parts)
    if c["act"] != "none":
        gate = p[:, :n]
        if c["act"] == "silu":
            gate = gate * torch.sigmoid(gate)
        else:
            gate = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)))
        p = gate * p[:, n:]
    return {"d": p}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4":
        return _exact_w4(s)
    return _exact_route(s) if case["op"].startswith("route") else _exact_rows(s)
