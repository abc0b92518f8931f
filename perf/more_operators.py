"""Measured cases of the operators around an 8-bit base model: the residual's addition with the
root-mean-square norm, and the gated activation, each with its rows left in 8-bit integers with a
scale per row, and the products of such rows with 8-bit weights that have a scale per channel.

`run` computes an operator in elementary torch operations (own = False) or through the
library's entry points (own = True); `exact` is its definition in 64 bits.

A row y in 8 bits: scale = max |y| / 127, codes = rint(y / scale) (ties to even), and a code c
stands for scale * c.  Both operators return what the codes stand for, in the 16 bits in which
the adapters of the layer read it."""
import torch

own = False

# (N, K) of the projections of one call, at the widths this repository is configured for
PROJ = {"7b-o": [(4096, 4096)], "7b-qkv": [(4096, 4096)] * 3, "13b-qkv": [(5120, 5120)] * 3,
        "8b-qkv": [(4096, 4096), (1024, 4096), (1024, 4096)], "8b-gate-up": [(14336, 4096)] * 2, "8b-down": [(4096, 14336)]}
EPS = 1e-5
# the most that a drawn case costs: multiplications of a product, values of a norm or an activation
MOST_PRODUCT, MOST_VALUES = 2011 * 28672 * 4096, 8191 * 4096


def listed():
    return [
        # one request's hidden row before its q, k and v: latency only
        {"name": "norm-one", "op": "norm", "rows": 1, "width": 4096, "add": True},
        # a decode step of 64 requests
        {"name": "norm-decode-64", "op": "norm", "rows": 64, "width": 5120, "add": True},
        # a step that is full of prompts, an odd number of rows
        {"name": "norm-prompts", "op": "norm", "rows": 8191, "width": 4096, "add": True},
        # one request's attention output, before the output projection
        {"name": "quantise-one", "op": "gate", "rows": 1, "width": 4096, "act": "none", "gated": False},
        # the MLP of a decode step of 64 requests
        {"name": "gate-decode-64", "op": "gate", "rows": 64, "width": 14336, "act": "silu", "gated": True},
        # the MLP of a step that is full of prompts
        {"name": "gate-prompts", "op": "gate", "rows": 2339, "width": 14336, "act": "silu", "gated": True},
        # one request: the output projection
        {"name": "product-one", "op": "product", "proj": "7b-o", "n": 0, "k": 0, "rows": 1},
        # a small decode batch: q, k and v of different widths in one call
        {"name": "product-qkv-13", "op": "product", "proj": "8b-qkv", "n": 0, "k": 0, "rows": 13},
        # a full decode batch: the two wide projections of the MLP
        {"name": "product-mlp-64", "op": "product", "proj": "8b-gate-up", "n": 0, "k": 0, "rows": 64},
        # a large decode batch with a few short prompts: q, k and v
        {"name": "product-qkv-200", "op": "product", "proj": "13b-qkv", "n": 0, "k": 0, "rows": 200},
        # a chunk of a prompt beside a decode batch: the long sums of the MLP's last projection
        {"name": "product-down-700", "op": "product", "proj": "8b-down", "n": 0, "k": 0, "rows": 700},
        # a step that is full of prompts
        {"name": "product-prompts", "op": "product", "proj": "8b-gate-up", "n": 0, "k": 0, "rows": 2011},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "gate", "product", "product"])
    if op == "product":
        proj = rng.choice(sorted(PROJ) + ["odd", "odd"])       # a model's projections, or one of any widths
        n, k = (8 * _log_int(rng, 8, 1800), 16 * _log_int(rng, 8, 900)) if proj == "odd" else (0, 0)
        each = sum(a * b for a, b in _shapes({"proj": proj, "n": n, "k": k}))
        return {"op": op, "proj": proj, "n": n, "k": k, "rows": _log_int(rng, 1, min(4096, MOST_PRODUCT // each))}
    width = rng.choice([4096, 5120, 14336, 16 * _log_int(rng, 4, 1024)])
    case = {"op": op, "rows": _log_int(rng, 1, min(16384, MOST_VALUES // width)), "width": width}
    if op == "norm":
        return {**case, "add": rng.random() < 0.75}
    return {**case, "act": rng.choice(["silu", "silu", "gelu", "gelu-tanh", "none"]), "gated": rng.random() < 0.75}


def _shapes(case):
    return [(case["n"], case["k"])] if case["proj"] == "odd" else PROJ[case["proj"]]


def work(case):
    t = case["rows"]
    if case["op"] == "product":
        b, f = 0, 0
        for k in {k for _, k in _shapes(case)}:
            b += t * k + 4 * t                                 # the projections read the same rows
        for n, k in _shapes(case):
            b += n * k + 4 * n + 2 * t * n
            f += 2 * t * n * k
        return {"bytes": b, "flops": f}
    # 16-bit rows read and written, codes and scales written
    d = case["width"]
    if case["op"] == "norm":
        return {"bytes": t * d * (2 + (4 if case["add"] else 0) + 3) + 4 * t + 2 * d, "flops": 6 * t * d}
    return {"bytes": t * d * (2 + (2 if case["gated"] else 0) + 3) + 4 * t, "flops": 8 * t * d}


# ---------------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t = case["rows"]
    s = {"op": case["op"], "rows": t}
    if case["op"] == "product":
        xs = {}
        for k in sorted({k for _, k in _shapes(case)}):
            # rows in 8 bits as the operators below leave them, and the scales of rows of unlike sizes
            x = _normal(g, t, k)
            top = x.abs().amax(1, keepdim=True)
            xs[k] = (torch.round(x * (127.0 / top)).to(torch.int8), (top[:, 0] / 127.0 * torch.exp(0.5 * _normal(g, t))).contiguous())
        s["w"] = []
        for n, k in _shapes(case):
            w = torch.round(_normal(g, n, k) * 33.0).clamp_(-127, 127).to(torch.int8)
            s["w"].append({"x": xs[k][0], "x_scales": xs[k][1], "w": w, "n": n, "k": k,
                           "w_scales": (0.5 + torch.rand(n, generator=g, device="cuda")) * (0.03 / k ** 0.5)})
        return s
    d = s["width"] = case["width"]
    if case["op"] == "norm":
        # a residual stream whose channels differ, what a layer adds to it, and the norm's weights
        channel = torch.exp(0.4 * _normal(g, d))
        s["x"] = (_normal(g, t, d) * 0.5).bfloat16()
        s["residual"] = (_normal(g, t, d) * channel * 2.0).bfloat16() if case["add"] else None
        s["weight"] = (0.5 + 0.1 * _normal(g, d)).bfloat16()
        return s
    s["act"] = case["act"]
    # the gate's and the other projection's outputs side by side, as one buffer holds them
    both = _normal(g, t, 2 * d if case["gated"] else d).bfloat16()
    s["gate"], s["up"] = both[:, :d], both[:, d:] if case["gated"] else None
    return s


# ---------------------------------------------------------------------------- the plain forms

def _codes(y):
    """Rows y f32 in 8 bits: the codes (as f32) and the scales."""
    top = y.abs().amax(1, keepdim=True)
    # a quotient next to a half needs 64 bits to fall on its side of it
    return torch.round(127.0 * y.double() / torch.where(top > 0, top, 1.0).double()).float(), top[:, 0] / 127.0


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    total = x.bfloat16()
    x = total.float()
    p = x * s["weight"].float()
    over = torch.rsqrt((x * x).mean(1) + EPS)
    codes, scale = _codes(p)                                   # the codes do not depend on the row's size, its scale does
    scale = scale * over
    out = {"x": (codes * scale[:, None]).bfloat16(), "scale": scale}
    if s["residual"] is not None:
        out["sum"] = total
    return out


def _plain_gate(s):
    a = s["gate"].float()
    if s["act"] == "silu":
        a = a / (1.0 + torch.exp(-a))
    elif s["act"] == "gelu":
        a = 0.5 * a * (1.0 + torch.erf(a * 0.5 ** 0.5))
    elif s["act"] == "gelu-tanh":
        a = 0.5 * a * (1.0 + torch.tanh((2.0 / torch.pi) ** 0.5 * (a + 0.044715 * a * a * a)))
    if s["up"] is not None:
        a = a * s["up"].float()
    codes, scale = _codes(a)
    return {"x": (codes * scale[:, None]).bfloat16(), "scale": scale}


def _plain_product(s):
    return [((w["x"].float() @ w["w"].float().t()) * w["x_scales"][:, None] * w["w_scales"]).bfloat16() for w in s["w"]]


# ---------------------------------------------------------------------------- the library's calls

def _kept(s):
    """What a serving program makes once and keeps beside its buffers: descriptions, workspace, output buffers."""
    if "kept" in s:
        return s["kept"]
    import heterogeneous_adapters_gb300 as lora
    t, kept = s["rows"], {"lora": lora}
    if s["op"] == "product":
        kept["y"] = [torch.empty(t, w["n"], dtype=torch.bfloat16, device="cuda") for w in s["w"]]
        kept["call"] = lora.w8_problems([(w["x"], w["x_scales"], y, w["k"], w["n"], w["w"], w["w_scales"], w["n"], w["k"])
                                         for w, y in zip(s["w"], kept["y"])])
        kept["size"] = lora.w8_workspace_size(kept["call"], t)
        kept["ws"] = torch.empty(kept["size"], dtype=torch.uint8, device="cuda")
        lora.kv_workspace_init(kept["ws"], kept["size"], torch.cuda.current_stream().cuda_stream)
    else:
        d = s["width"]
        x = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
        codes, scales = torch.empty(t, d, dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
        rows = lora.Q8Rows(codes, d, scales, x, d, lora.LORA_Q8_X_HELD)
        kept["out"] = {"x": x, "scale": scales}
        if s["op"] == "norm":
            total = torch.empty_like(x) if s["residual"] is not None else None
            kept["call"] = lora.Q8Norm(s["x"], d, s["residual"], d, total, d, s["weight"], EPS, d, rows)
            if total is not None:
                kept["out"]["sum"] = total
        else:
            act = {"none": lora.LORA_ACT_NONE, "silu": lora.LORA_ACT_SILU, "gelu": lora.LORA_ACT_GELU, "gelu-tanh": lora.LORA_ACT_GELU_TANH}
            kept["call"] = lora.Q8Gate(s["gate"], s["gate"].stride(0), s["up"], s["gate"].stride(0), act[s["act"]], d, rows)
    s["kept"] = kept
    return kept


def _own(s):
    kept = _kept(s)
    lora, stream = kept["lora"], torch.cuda.current_stream().cuda_stream
    if s["op"] == "product":
        lora.w8_matmul(kept["call"], s["rows"], kept["ws"], kept["size"], stream)
        return kept["y"]
    (lora.q8_norm if s["op"] == "norm" else lora.q8_gate)(kept["call"], s["rows"], stream)
    return kept["out"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "gate": _plain_gate, "product": _plain_product}[state["op"]](state)


# ---------------------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(y, step):
    """What 8 bits hold of rows y f64, whose scales are `step` (64 bits)."""
    return torch.where(step > 0, torch.round(y / torch.where(step > 0, step, 1.0)), 0.0) * step


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "product":
        out = []
        for w in s["w"]:
            x = w["x"].double() * w["x_scales"].double()[:, None]
            out.append(x @ (w["w"].double() * w["w_scales"].double()[:, None]).T)
        return out
    if s["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).bfloat16().double()   # the stream is held in 16 bits
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / s["width"] + EPS) * s["weight"].double()
    else:
        y = s["gate"].double()
        if s["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif s["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif s["act"] == "gelu-tanh":
            y = y * torch.sigmoid(2.0 * (2.0 / torch.pi) ** 0.5 * (y + 0.044715 * y.pow(3)))
        if s["up"] is not None:
            y = y * s["up"].double()
    step = y.abs().max(1, keepdim=True).values / 127
    out = {"x": _exact_rows(y, step), "scale": step[:, 0]}
    if s["op"] == "norm" and s["residual"] is not None:
        out["sum"] = h
    return out
