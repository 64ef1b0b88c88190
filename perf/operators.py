"""Measured cases of the operators around the compressed products of a
transformer block: the RMS norm with the residual's addition, the product with
bias, activation and residual in its epilogue, and the gated feed-forward
product, each with its backward pass.

The weights are frozen and kept compressed (DF11, MFMA tile order), so the
backward passes give the gradients of the activations, the biases, the
residual and the norm's weight.  Where `own` is false the operators run in
their plain form, elementary torch operations in 32 bits on the BF16 weights.

    norm    s = round(x + residual)  (x itself without a residual)
            y = s * rsqrt(mean(s^2) + eps) * weight
    product y = act(x W^T + bias) + residual
    gated   h = act(x Wg^T + bg) * (x Wu^T + bu)
"""

import math

import torch

own = False

EPS = 1e-5

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# Stored bits of one weight: sign and mantissa verbatim, about 2.6 bits of
# exponent entropy.
WEIGHT_BYTES = 10.6 / 8


def _case(op, name, **more):
    case = {"op": op, "tokens": 1, "cols": 4096, "rows": 4096, "type": "bf16", "out": "bf16", "act": "none",
            "bias": False, "residual": False, "weight": True, "grad": False}
    case.update(more)
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # One token of decoding between two projections: the call's latency.
        _case("norm", "norm_one_token", residual=True),
        # A long prompt's activations.
        _case("norm", "norm_prompt", tokens=8192, residual=True),
        # Float activations whose width is odd: no two rows are aligned alike.
        _case("norm", "norm_odd_width", tokens=333, cols=5003, type="fp32"),
        # A training step's norm: both outputs carry gradients.
        _case("norm", "norm_grad", tokens=2048, residual=True, grad=True),
        # The down projection of one token, added to the residual stream.
        _case("product", "product_one_token", cols=14336, residual=True),
        # A ragged batch of requests in a float result with bias and GELU.
        _case("product", "product_odd_batch", tokens=37, bias=True, act="gelu", out="fp32"),
        # The output projection of a prompt, added to the residual stream.
        _case("product", "product_prompt", tokens=2048, residual=True),
        # An adapter's training step through a frozen projection.
        _case("product", "product_grad", tokens=777, rows=1024, bias=True, act="gelu_tanh", residual=True,
              grad=True),
        # Gate and up of one token, the largest weights of a block.
        _case("gated", "gated_one_token", rows=14336, act="silu"),
        # Gate and up of a serving batch.
        _case("gated", "gated_batch", tokens=64, rows=14336, act="silu"),
        # Gate and up of a prompt whose length fits no tile.
        _case("gated", "gated_prompt", tokens=1999, rows=14336, act="silu"),
        # A training step through the frozen feed-forward block.
        _case("gated", "gated_grad", tokens=1024, rows=14336, act="silu", grad=True),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["norm", "product", "gated"])
    if op == "norm":
        cols = _spread(rng, 128, 16384)
        return _case(op, None, tokens=_spread(rng, 1, min(8192, 8192 * 4096 // cols)), cols=cols,
                     type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), residual=rng.random() < 0.6,
                     weight=rng.random() < 0.8, grad=rng.random() < 0.4)
    cols, rows = 32 * _spread(rng, 8, 448), 64 * _spread(rng, 4, 224)
    while cols * rows > 4096 * 14336:
        cols, rows = 32 * _spread(rng, 8, 448), 64 * _spread(rng, 4, 224)
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"] + (["none", "none"] if op == "product" else []))
    return _case(op, None, tokens=_spread(rng, 1, 1024), cols=cols, rows=rows, act=act,
                 out=rng.choice(["bf16", "bf16", "fp32"]), bias=rng.random() < 0.5,
                 residual=op == "product" and rng.random() < 0.5, grad=rng.random() < 0.4)


def _weights(g, rows, cols):
    """Trained-weight statistics: N(0, 0.02^2) with one entry in 10^4 an outlier from N(0, 1)."""
    w = torch.randn(rows, cols, device="cuda", generator=g)
    far = torch.rand(rows, cols, device="cuda", generator=g) < 1e-4
    return torch.where(far, w, w * 0.02).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t, c, r, kind = case["tokens"], case["cols"], case["rows"], TYPES[case["type"]]
    state = {"case": case}
    if case["op"] == "norm":
        state["x"] = torch.randn(t, c, device="cuda", generator=g).to(kind)
        if case["residual"]:
            state["residual"] = (3 * torch.randn(t, c, device="cuda", generator=g)).to(kind)
        if case["weight"]:
            state["weight"] = (1 + 0.2 * torch.randn(c, device="cuda", generator=g)).to(kind)
        if case["grad"]:
            state["dy"] = torch.randn(t, c, device="cuda", generator=g).to(kind)
            if case["residual"]:
                state["ds"] = torch.randn(t, c, device="cuda", generator=g).to(kind)
        return state
    state["x"] = torch.randn(t, c, device="cuda", generator=g).to(kind)
    ws = {n: _weights(g, r, c) for n in (("w",) if case["op"] == "product" else ("gate", "up"))}
    if case["bias"]:
        for n in ws:
            state[n + "_bias"] = (0.5 * torch.randn(r, device="cuda", generator=g)).to(kind)
    out = TYPES[case["out"]]
    if case["residual"]:
        state["residual"] = torch.randn(t, r, device="cuda", generator=g).to(out)
    if case["grad"]:
        state["dy"] = torch.randn(t, r, device="cuda", generator=g).to(out)
    if own:
        # A program keeps its weights compressed; they are compressed once.
        from entropy_decoding_df11_amd import df11
        ws = {n: df11.compress(w.cpu(), layout="mfma_tiles") for n, w in ws.items()}
    state.update(ws)
    return state


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "relu":
        return torch.clamp(z, min=0)
    return z


def _slope(name, z):
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        u = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * k * (1 + 3 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _plain_norm(s):
    kind, case, out = s["x"].dtype, s["case"], {}
    total = s["x"]
    if case["residual"]:
        total = out["sum"] = (s["x"].float() + s["residual"].float()).to(kind)
    f = total.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    w = s["weight"].float() if case["weight"] else torch.ones_like(f[0])
    out["y"] = (f * r * w).to(kind)
    if case["grad"]:
        dy, hat = s["dy"].float(), f * r
        d = dy * w
        dx = r * (d - hat * (d * hat).mean(-1, keepdim=True))
        if case["residual"]:
            dx = dx + s["ds"].float()
        out["dx"] = dx.to(kind)
        if case["weight"]:
            out["dweight"] = (dy * hat).sum(0).to(kind)
    return out


def _plain_linear(s, n):
    z = s["x"].float() @ s[n].float().t()
    return z + s[n + "_bias"].float() if s["case"]["bias"] else z


def _plain_product(s):
    case = s["case"]
    z = _plain_linear(s, "w")
    y = _act(case["act"], z)
    if case["residual"]:
        y = y + s["residual"].float()
    out = {"y": y.to(TYPES[case["out"]])}
    if case["grad"]:
        dz = s["dy"].float() * _slope(case["act"], z)
        out["dx"] = (dz @ s["w"].float()).to(s["x"].dtype)
        if case["bias"]:
            out["dbias"] = dz.sum(0).to(s["w_bias"].dtype)
    return out


def _plain_gated(s):
    case = s["case"]
    zg, zu = _plain_linear(s, "gate"), _plain_linear(s, "up")
    a = _act(case["act"], zg)
    out = {"y": (a * zu).to(TYPES[case["out"]])}
    if case["grad"]:
        dy = s["dy"].float()
        dg, du = dy * zu * _slope(case["act"], zg), dy * a
        out["dx"] = (dg @ s["gate"].float() + du @ s["up"].float()).to(s["x"].dtype)
        if case["bias"]:
            out["dgate_bias"] = dg.sum(0).to(s["gate_bias"].dtype)
            out["dup_bias"] = du.sum(0).to(s["up_bias"].dtype)
    return out


def _leaf(t, wanted):
    return t.detach().requires_grad_() if wanted and t is not None else t


def _own_norm(s):
    from entropy_decoding_df11_amd import df11
    case = s["case"]
    x, w = _leaf(s["x"], case["grad"]), _leaf(s.get("weight"), case["grad"])
    got = df11.rms_norm(x, weight=w, residual=s.get("residual"), eps=EPS)
    out = {"y": got}
    if case["residual"]:
        out = {"sum": got[1], "y": got[0]}
    if case["grad"]:
        tops = (out["y"], out["sum"]) if case["residual"] else (out["y"],)
        downs = (s["dy"], s["ds"]) if case["residual"] else (s["dy"],)
        grads = torch.autograd.grad(tops, (x, w) if case["weight"] else (x,), downs)
        out.update(zip(("dx", "dweight"), grads))
    return out


def _own_product(s):
    from entropy_decoding_df11_amd import df11
    case = s["case"]
    x, b = _leaf(s["x"], case["grad"]), _leaf(s.get("w_bias"), case["grad"])
    out = {"y": df11.matmul_epilogue(s["w"], x, bias=b, activation=case["act"], residual=s.get("residual"),
                                     out_dtype=TYPES[case["out"]])}
    if case["grad"]:
        out.update(zip(("dx", "dbias"), torch.autograd.grad(out["y"], (x, b) if case["bias"] else (x,), s["dy"])))
    return out


def _own_gated(s):
    from entropy_decoding_df11_amd import df11
    case = s["case"]
    x, bg, bu = (_leaf(s.get(n), case["grad"]) for n in ("x", "gate_bias", "up_bias"))
    out = {"y": df11.gated_matmul(s["gate"], s["up"], x, gate_bias=bg, up_bias=bu, activation=case["act"],
                                  out_dtype=TYPES[case["out"]])}
    if case["grad"]:
        grads = torch.autograd.grad(out["y"], (x, bg, bu) if case["bias"] else (x,), s["dy"])
        out.update(zip(("dx", "dgate_bias", "dup_bias"), grads))
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "product": _own_product, "gated": _own_gated}[op](state)
    return {"norm": _plain_norm, "product": _plain_product, "gated": _plain_gated}[op](state)


def work(case):
    t, c, r = case["tokens"], case["cols"], case["rows"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "norm":
        each = size[case["type"]]
        rows = 2 + 2 * case["residual"]  # x and y, the residual and the sum
        if case["grad"]:
            rows += 2 + case["residual"]  # dy and dx, the sum's gradient
        vectors = case["weight"] * (1 + case["grad"])
        return {"bytes": each * (t * c * rows + c * vectors), "flops": t * c * (12 if case["grad"] else 5)}
    n, out = 1 + (case["op"] == "gated"), size[case["out"]]
    # x, the compressed weights, the biases, the residual and the output
    total = 2 * t * c + n * (WEIGHT_BYTES * r * c + 2 * r * case["bias"]) + out * t * r * (1 + case["residual"])
    flops = 2 * n * t * r * c
    if case["grad"]:  # dy, dx, the weights again, the biases' gradients
        total += out * t * r + 2 * t * c + n * (WEIGHT_BYTES * r * c + 2 * r * case["bias"])
        flops *= 2
    return {"bytes": int(total), "flops": flops}


def _act64(name, z):
    """(value, slope) in 64 bits."""
    if name == "silu":
        p = 0.5 + 0.5 * torch.tanh(0.5 * z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        v = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(v)
        return z * p, p + z * p * torch.sigmoid(-v) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z.square())
    if name == "relu":
        return z.relu(), (z > 0).double()
    return z, torch.ones_like(z)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    d = {k: v.double() for k, v in s.items() if k != "case"}
    if case["op"] == "norm":
        out, kind = {}, TYPES[case["type"]]
        v = d["x"]
        if case["residual"]:
            v = out["sum"] = (d["x"] + d["residual"]).to(kind).double()
        scale = (v.square().sum(1) / v.shape[1] + EPS).pow(-0.5)
        unit = v * scale[:, None]
        w = d.get("weight", torch.ones(v.shape[1], dtype=torch.float64, device=v.device))
        out["y"] = unit * w
        if case["grad"]:
            wdy = d["dy"] * w
            inner = (wdy * unit).sum(1) / v.shape[1]
            out["dx"] = (wdy - unit * inner[:, None]) * scale[:, None] + d.get("ds", 0.0)
            if case["weight"]:
                out["dweight"] = (unit * d["dy"]).sum(0)
        return out
    names = ("w",) if case["op"] == "product" else ("gate", "up")
    z = [torch.mm(d[n], d["x"].t()) for n in names]  # rows x tokens
    if case["bias"]:
        z = [v + d[n + "_bias"][:, None] for v, n in zip(z, names)]
    value, slope = _act64(case["act"], z[0])
    y = value * z[1] if case["op"] == "gated" else value
    out = {"y": y.t() + d["residual"] if case["residual"] else y.t().contiguous()}
    if case["grad"]:
        dy = d["dy"].t()
        dz = [dy * slope] if case["op"] == "product" else [dy * slope * z[1], dy * value]
        out["dx"] = sum(torch.mm(d[n].t(), v) for n, v in zip(names, dz)).t().contiguous()
        if case["bias"]:
            out.update({"d" + (n + "_bias" if len(names) > 1 else "bias"): v.sum(1) for n, v in zip(names, dz)})
    return out
