"""The 8-bit operators, their plain forms and the cases that they are measured on.

The operators: a root-mean-square norm with the residual's addition and 8-bit rows out, the
quantisation of rows (as they are, or of silu(gate) * up) and of filters, reading 8-bit rows back, the
matrix product of 8-bit rows and filters, and the 1 x 1 convolution that is made of them. With
`own` false run() computes them in elementary torch operations.
"""
import math

import torch

own = False
EPS = 1e-6


def listed():
    return [
        # one token of a decoding step: the time of the launches
        {"name": "norm, one token", "op": "norm", "m": 1, "c": 4096, "dtype": "bf16", "residual": True},
        # a batch of prompts
        {"name": "norm, prompts", "op": "norm", "m": 8192, "c": 4096, "dtype": "bf16", "residual": True},
        # a ragged batch of an odd width in single precision
        {"name": "norm, odd f32", "op": "norm", "m": 1031, "c": 5003, "dtype": "f32", "residual": False},
        # the frames of 16 audio clips between two layers of a Conv1D stem (width 512)
        {"name": "rows, audio frames", "op": "rows", "m": 48000, "c": 512, "dtype": "bf16", "glu": False},
        # the gated activations of a feed-forward pair, a ragged batch
        {"name": "rows, gated", "op": "rows", "m": 1999, "c": 10240, "dtype": "bf16", "glu": True},
        # the filter of a small pointwise layer, and a large projection's, once when a network is loaded
        {"name": "filter, pointwise", "op": "filter", "c": 256, "n": 512, "dtype": "bf16"},
        {"name": "filter, projection", "op": "filter", "c": 4096, "n": 16384, "dtype": "bf16"},
        # one token through a square projection: the filter's bytes
        {"name": "product, one token", "op": "product", "m": 1, "c": 4096, "n": 4096, "dtype": "bf16", "bias": False},
        # a small ragged batch, odd in every size, with a bias, in single precision
        {"name": "product, odd", "op": "product", "m": 301, "c": 5003, "n": 4999, "dtype": "f32", "bias": True},
        # prompts through a wide projection: the tensor cores' rate
        {"name": "product, prompts", "op": "product", "m": 16384, "c": 4096, "n": 16384, "dtype": "bf16", "bias": False},
        # the pointwise layer of the benchmark: 32 images of 28 x 28, 256 -> 512 channels
        {"name": "layer, pointwise", "op": "layer", "batch": 32, "h": 28, "w": 28, "c": 256, "n": 512, "norm": False, "bias": True},
        # norm and projection of 512 tokens
        {"name": "layer, tokens", "op": "layer", "batch": 1, "h": 1, "w": 512, "c": 4096, "n": 4096, "norm": True, "bias": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    c = _log(rng, lo, hi)
    return c if rng.random() < 0.4 else max(lo, c // 64 * 64)  # most widths are whole, some odd


def draw(rng):
    op = rng.choice(["norm", "rows", "filter", "product", "product", "layer"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        c = _width(rng, 64, 16384)
        return {"op": op, "m": _log(rng, 1, (1 << 25) // c), "c": c, "dtype": dtype, "residual": rng.random() < 0.6}
    if op == "rows":
        c = _width(rng, 64, 16384)
        return {"op": op, "m": _log(rng, 1, (1 << 24) // c), "c": c, "dtype": dtype, "glu": rng.random() < 0.5}
    if op == "filter":
        return {"op": op, "c": _width(rng, 64, 8192), "n": _width(rng, 64, 8192), "dtype": dtype}
    c, n = _width(rng, 64, 8192), _width(rng, 64, 16384)
    if op == "product":
        m = _log(rng, 1, min(16384, (1 << 39) // (c * n)))
        return {"op": op, "m": m, "c": c, "n": n, "dtype": dtype, "bias": rng.random() < 0.5}
    batch, h = rng.choice([(1, 1), (8, 7), (8, 14), (32, 14)])
    w = _log(rng, 1, 4096) if h == 1 else h
    return {"op": op, "batch": batch, "h": h, "w": w, "c": min(c, 4096), "n": min(n, 4096), "norm": rng.random() < 0.5, "bias": rng.random() < 0.5}


def _type(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _scaled(t):
    """8-bit rows of t and their scales; rows start on a 16-byte boundary, as the framework lays them out."""
    a = t.abs().amax(-1, keepdim=True).clamp_min(1e-30)
    m, c = t.shape
    q = torch.zeros(m, (c + 15) // 16 * 16, dtype=torch.int8, device=t.device)[:, :c]
    q.copy_((t * (127 / a)).round())
    return q, (a / 127).reshape(-1)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def tokens(m, c):
        # a few channels of a network's tokens are far larger than the others
        return normal(m, c) * (1 + 19 * (torch.rand(c, generator=g, device="cuda") < 0.01))

    s, op, t, c = {"case": case}, case["op"], _type(case), case["c"]
    if op == "norm":
        s["x"] = tokens(case["m"], c).to(t)
        s["residual"] = tokens(case["m"], c).to(t) if case["residual"] else None
        s["weight"] = 1 + 0.2 * normal(c)
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"] = torch.empty(case["m"], c, dtype=torch.bfloat16, device="cuda")
    elif op == "rows":
        s["x"] = tokens(case["m"], 2 * c if case["glu"] else c).to(t)
        s["y"] = torch.empty(case["m"], c, dtype=torch.bfloat16, device="cuda")
    elif op == "filter":
        s["filter"] = (normal(c, case["n"]) / math.sqrt(c)).to(t)
        s["y"] = torch.empty(case["n"], c, dtype=torch.bfloat16, device="cuda")
    else:
        n = case["n"]
        s["wq"], s["ws"] = _scaled(normal(n, c) / math.sqrt(c))
        s["bias"] = 0.3 * normal(n) if case["bias"] else None
        if op == "product":
            s["q"], s["qs"] = _scaled(tokens(case["m"], c))
            s["y"] = torch.empty(case["m"], n, dtype=t, device="cuda")
        else:
            shape = case["batch"], case["h"], case["w"]
            s["x"] = tokens(math.prod(shape), c).to(t).reshape(*shape, c)
            s["weight"] = 1 + 0.2 * normal(c) if case["norm"] else None
            s["y"] = torch.empty(*shape, n, dtype=t, device="cuda")
            s["workspace"] = torch.empty(math.prod(shape) * ((c + 15) // 16 * 16 + 4) + 16, dtype=torch.uint8, device="cuda")
    if op in ("norm", "rows", "filter"):
        rows, width = s["y"].shape
        s["q"] = torch.empty(rows, (width + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :width]
        s["qs"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    return s


def _own(s):
    import cnn_convolution_nhwc_b200 as cb

    case = s["case"]
    op = case["op"]
    if op == "product":
        return cb.pointwise_i8_fwd(s["q"], s["qs"], s["wq"], s["ws"], s["bias"], y=s["y"])
    if op == "layer":
        return cb.conv2d_nhwc_fwd_i8(s["x"], s["wq"], s["ws"], s["bias"], norm=s["weight"], eps=EPS, Y=s["y"], workspace=s["workspace"])
    if op == "norm":
        q, scale, h = cb.rmsnorm_i8_fwd(s["x"], s["weight"], s["residual"], eps=EPS, q=s["q"], scale=s["qs"], h=s["h"])
        y = cb.dequant_rows_i8_fwd(q, scale, y=s["y"])
        return (y, scale, h) if case["residual"] else (y, scale)
    if op == "rows":
        q, scale = cb.quant_rows_i8_fwd(s["x"], glu=case["glu"], q=s["q"], scale=s["qs"])
    else:
        q, scale = cb.quant_filter_i8_fwd(s["filter"], q=s["q"], scale=s["qs"])
    return cb.dequant_rows_i8_fwd(q, scale, y=s["y"]), scale


def _rows(t):
    """The 8-bit values of rows and the largest magnitudes. 127 t / a is rounded in 64 bits: it can lie at the border of two values."""
    a = t.abs().amax(-1, keepdim=True)
    return torch.where(a > 0, t.double() * 127 / a.double(), 0.0).round().float(), a


def _norm(x, residual, weight):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    rstd = 1 / (h.float().square().mean(-1, keepdim=True) + EPS).sqrt()
    q, a = _rows(h.float() * weight)
    return q, a * rstd / 127, h


def _product(q, scale, wq, ws, bias, t):
    y = (q.float() @ wq.float().t()) * scale * ws
    return (y if bias is None else y + bias).to(t)


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    op, t = case["op"], _type(case)
    if op == "norm":
        q, scale, h = _norm(s["x"], s["residual"], s["weight"])
        y = (q * scale).bfloat16(), scale.reshape(-1)
        return (*y, h) if case["residual"] else y
    if op == "rows":
        v, c = s["x"].float(), case["c"]
        if case["glu"]:
            v = v[:, :c] / (1 + (-v[:, :c]).exp()) * v[:, c:]
        q, a = _rows(v)
        return (q * (a / 127)).bfloat16(), (a / 127).reshape(-1)
    if op == "filter":
        q, a = _rows(s["filter"].float().t().contiguous())
        return (q * (a / 127)).bfloat16(), (a / 127).reshape(-1)
    if op == "product":
        return _product(s["q"], s["qs"][:, None], s["wq"], s["ws"], s["bias"], t)
    x = s["x"].reshape(-1, case["c"])
    if case["norm"]:
        q, scale, _ = _norm(x, None, s["weight"])
    else:
        q, a = _rows(x.float())
        scale = a / 127
    return _product(q, scale, s["wq"], s["ws"], s["bias"], t).reshape(*s["x"].shape[:3], case["n"])


def work(case):
    op, c, e = case["op"], case["c"], 4 if case.get("dtype") == "f32" else 2
    if op in ("norm", "rows"):
        m = case["m"]
        read = (2 if case.get("residual") or case.get("glu") else 1) * m * c * e
        wrote = m * c * (2 + (e if case.get("residual") else 0)) + 4 * m
        return {"bytes": read + wrote + (4 * c if op == "norm" else 0), "flops": 10 * m * c}
    n = case["n"]
    if op == "filter":
        return {"bytes": c * n * (e + 2) + 4 * n, "flops": 4 * c * n}
    m = case["m"] if op == "product" else case["batch"] * case["h"] * case["w"]
    read = m * c + 4 * m if op == "product" else 2 * m * c + (4 * c if case["norm"] else 0)
    return {"bytes": read + n * c + 4 * n + (4 * n if case["bias"] else 0) + m * n * e, "flops": 2 * m * n * c}


def exact(case, seed):
    s, op, c = prepare(case, seed), case["op"], case["c"]
    of = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("y", "h", "workspace")}

    def levels(v, gain=1.0):
        top = torch.linalg.vector_norm(v, ord=math.inf, dim=1, keepdim=True)
        whole = torch.where(top > 0, v * (127 / top), torch.zeros_like(v)).round()
        return whole, top * gain / 127

    if op in ("norm", "layer"):
        h = of["x"].reshape(-1, c)
        if op == "norm" and case["residual"]:
            h = (h + of["residual"]).to(s["x"].dtype).double()  # the sum is held in the tokens' type
        if op == "norm" or case["norm"]:
            whole, step = levels(h * of["weight"], torch.rsqrt((h * h).sum(1, keepdim=True) / c + EPS))
        else:
            whole, step = levels(h)
        if op == "norm":
            return (whole * step, step[:, 0], h) if case["residual"] else (whole * step, step[:, 0])
    elif op == "rows":
        v = of["x"] if not case["glu"] else torch.sigmoid(of["x"][:, :c]) * of["x"][:, :c] * of["x"][:, c:]
        whole, step = levels(v)
        return whole * step, step[:, 0]
    elif op == "filter":
        whole, step = levels(of["filter"].T)
        return whole * step, step[:, 0]
    else:
        whole, step = of["q"], of["qs"].unsqueeze(1)
    y = torch.einsum("mc,nc->mn", whole * step, of["wq"] * of["ws"].unsqueeze(1))
    if case["bias"]:
        y += of["bias"]
    return y.reshape(s["y"].shape)
