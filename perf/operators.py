"""Measured cases of the decode-step operators around the multi-LoRA delta: appending keys and
values to a paged 4-bit cache (rotary positions applied on the way), attention over that
cache, and products with 4-bit weights.

`run` computes an operator in elementary torch operations (own = False) or through the
library's entry points (own = True); `exact` is its definition in 64 bits.

The 4-bit cache.  A block holds `block` tokens of every KV head, as tiles of 16 tokens of one
head: [kv head][block / 16] tiles.  A tile is K codes [D / 32][16 tokens][16 bytes], V codes
likewise, K parameters [D / group][16 tokens] of (f16 scale, f16 offset), V parameters
likewise; a byte holds two neighbouring dimensions, the even one in its low half, and a code c
stands for scale * (c - 8) + offset."""
import numpy as np
import torch

own = False

# (query heads, KV heads, head dimension, layer width) of the models this repository is
# configured for, and a small one with narrow heads
HEADS = {"7b": (32, 32, 128), "13b": (40, 40, 128), "8b": (32, 8, 128), "narrow": (16, 4, 64)}
# (N, K) of the projections of one call
PROJ = {"7b-o": [(4096, 4096)], "7b-qkv": [(4096, 4096)] * 3, "13b-qkv": [(5120, 5120)] * 3,
        "8b-qkv": [(4096, 4096), (1024, 4096), (1024, 4096)], "8b-kv": [(1024, 4096)] * 2,
        "8b-gate-up": [(14336, 4096)] * 2, "8b-down": [(4096, 14336)]}


def listed():
    return [
        # one request: its token's keys and values, latency only
        {"name": "append-one", "op": "append", "model": "8b", "seqs": 1, "q_lo": 1, "q_hi": 1, "len_lo": 1000, "len_hi": 1000,
         "group": 128, "block": 32, "pairs": False, "lens": 1},
        # a decode step of 64 requests, one scale per 32 values
        {"name": "append-decode-64", "op": "append", "model": "7b", "seqs": 64, "q_lo": 1, "q_hi": 1, "len_lo": 1, "len_hi": 4000,
         "group": 32, "block": 16, "pairs": False, "lens": 2},
        # prompts of odd lengths, written whole
        {"name": "append-prompts", "op": "append", "model": "8b", "seqs": 8, "q_lo": 129, "q_hi": 2047, "len_lo": 2100,
         "len_hi": 4000, "group": 128, "block": 64, "pairs": True, "lens": 3},
        # one request in the middle of its answer
        {"name": "attend-one", "op": "attend", "model": "8b", "seqs": 1, "q_lo": 1, "q_hi": 1, "len_lo": 1237, "len_hi": 1237,
         "group": 128, "block": 32, "lens": 4},
        # a full decode batch, grouped-query heads, ragged contexts
        {"name": "attend-decode-64", "op": "attend", "model": "8b", "seqs": 64, "q_lo": 1, "q_hi": 1, "len_lo": 17, "len_hi": 8191,
         "group": 128, "block": 64, "lens": 5},
        # one query head per KV head, one scale per 32 values
        {"name": "attend-decode-mha", "op": "attend", "model": "7b", "seqs": 32, "q_lo": 1, "q_hi": 1, "len_lo": 100,
         "len_hi": 3001, "group": 32, "block": 16, "lens": 6},
        # few requests with long contexts: the work is split along the keys
        {"name": "attend-long", "op": "attend", "model": "8b", "seqs": 2, "q_lo": 1, "q_hi": 1, "len_lo": 100001, "len_hi": 131071,
         "group": 128, "block": 64, "lens": 7},
        # several drafted tokens per request are checked at once, narrow heads
        {"name": "attend-verify", "op": "attend", "model": "narrow", "seqs": 48, "q_lo": 1, "q_hi": 5, "len_lo": 33, "len_hi": 4095,
         "group": 64, "block": 32, "lens": 8},
        # chunks of long prompts over what the cache already holds
        {"name": "attend-chunk", "op": "attend", "model": "8b", "seqs": 3, "q_lo": 300, "q_hi": 512, "len_lo": 3111, "len_hi": 6000,
         "group": 128, "block": 64, "lens": 9},
        # one request: the output projection
        {"name": "w4-one", "op": "w4", "proj": "7b-o", "rows": 1, "group": 128, "zeros": True},
        # a small batch: q, k and v of different widths in one call
        {"name": "w4-qkv-13", "op": "w4", "proj": "8b-qkv", "rows": 13, "group": 64, "zeros": True},
        # a full decode batch: the two wide projections of the MLP
        {"name": "w4-mlp-64", "op": "w4", "proj": "8b-gate-up", "rows": 64, "group": 128, "zeros": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "w4"])
    if op == "w4":
        return {"op": op, "proj": rng.choice(sorted(PROJ)), "rows": _log_int(rng, 1, 128), "group": rng.choice([32, 64, 128]),
                "zeros": rng.random() < 0.6}
    model = rng.choice(sorted(HEADS))
    heads, kv_heads, dim = HEADS[model]
    case = {"op": op, "model": model, "group": rng.choice([32, dim]), "block": rng.choice([16, 32, 64, 128]),
            "lens": rng.randrange(1 << 30)}
    if op == "append":
        rows = _log_int(rng, 1, 8000 * 8 // kv_heads)          # rows of the call, in requests of q rows or less
        q = 1 if rng.random() < 0.5 else _log_int(rng, 1, min(2047, rows))
        return {**case, "seqs": max(1, min(256, rows // q)), "q_lo": max(1, q // 3), "q_hi": q, "len_lo": q, "len_hi": q + _log_int(rng, 1, 4000),
                "pairs": rng.random() < 0.5}
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    if kind == "chunk":
        q, seqs, longest = _log_int(rng, 16, 448), rng.randint(1, 3), 3500 * 32 // heads
        return {**case, "seqs": seqs, "q_lo": max(1, q // 2), "q_hi": q, "len_lo": q, "len_hi": q + _log_int(rng, 1, longest)}
    seqs = _log_int(rng, 1, 128)
    longest = min(131071, 200000 * 8 // kv_heads // seqs)      # tokens of the call stay under a bound
    length = _log_int(rng, 16, longest)
    q = 1 if kind == "decode" else rng.randint(2, 8)
    return {**case, "seqs": seqs, "q_lo": 1, "q_hi": q, "len_lo": max(q, length // rng.choice([1, 3, 50])), "len_hi": max(q, length)}


# ---------------------------------------------------------------------------- shapes

def _lens(case):
    """(rows, cached tokens with them) of each request."""
    r = np.random.RandomState(case["lens"])
    q = r.randint(case["q_lo"], case["q_hi"] + 1, case["seqs"]).astype(np.int64)
    n = r.randint(case["len_lo"], case["len_hi"] + 1, case["seqs"]).astype(np.int64)
    return q, np.maximum(n, q)


def _token_bytes(dim, group):
    """Bytes of one token's keys and values of one head: codes, scales and offsets."""
    return dim + 8 * (dim // group)


def work(case):
    if case["op"] == "w4":
        t, b, f = case["rows"], 0, 0
        for k in {k for _, k in PROJ[case["proj"]]}:
            b += 2 * t * k                                     # x is the same rows for all projections
        for n, k in PROJ[case["proj"]]:
            b += n * k // 2 + n * (k // case["group"]) * 2 + (n * (k // case["group"]) // 2 if case["zeros"] else 0) + 2 * t * n
            f += 2 * t * n * k
        return {"bytes": b, "flops": f}
    heads, kv_heads, dim = HEADS[case["model"]]
    q, n = _lens(case)
    rows, tokens = int(q.sum()), int(n.sum())
    if case["op"] == "append":
        # q, k, v and the rotations read; q, the cache's tokens and the values they stand for written
        return {"bytes": rows * (2 * heads * dim * 2 + 2 * kv_heads * dim * 4 + kv_heads * _token_bytes(dim, case["group"]) + dim * 4),
                "flops": rows * (heads + kv_heads) * dim * 3}
    pairs = int((q * n - q * (q - 1) // 2).sum())
    return {"bytes": tokens * kv_heads * _token_bytes(dim, case["group"]) + rows * heads * (dim * 4 + 4),
            "flops": 4 * pairs * heads * dim}


# ---------------------------------------------------------------------------- the cache in torch

def _regions(s, blocks):
    """K codes, V codes, K and V parameters of the cache as views, each
    [blocks, kv heads, sub-tiles, chunks, 16 tokens, bytes]."""
    stride, hk, sub, dim, ng = s["stride"], s["kv_heads"], s["block"] // 16, s["dim"], s["dim"] // s["group"]
    tile, out, at = 16 * _token_bytes(s["dim"], s["group"]), [], 0
    for chunks, width in ((dim // 32, 16), (dim // 32, 16), (ng, 4), (ng, 4)):
        out.append(torch.as_strided(blocks, (blocks.numel() // stride, hk, sub, chunks, 16, width),
                                    (stride, sub * tile, tile, 16 * width, width, 1), at))
        at += chunks * 16 * width
    return out


def _quantise(x, group):
    """x f32 [.., D] -> code bytes [.., D / 32, 16] and parameter bytes [.., D / group, 4]."""
    g = x.reshape(*x.shape[:-1], -1, group)
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((hi - lo) * torch.tensor(1.0 / 15.0, device=x.device)).clamp(max=65504.0).half()
    wide = scale.float()
    offset = (lo + 8.0 * wide).clamp(-65504.0, 65504.0).half()
    inverse = torch.where(wide > 0, 1.0 / wide, torch.zeros_like(wide))
    c = (torch.round((g - offset.float()) * inverse).clamp(-8, 7) + 8).to(torch.uint8).reshape(*x.shape[:-1], -1, 16, 2)
    params = torch.cat([scale, offset], -1).contiguous().view(torch.uint8)
    return c[..., 0] | (c[..., 1] << 4), params


def _values(codes, params, group):
    """The values that code bytes [.., D / 32, 16] with parameter bytes [.., D / group, 4] stand for, f32 [.., D]."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-2], -1, group).float() - 8.0
    p = params.contiguous().view(torch.float16).float()
    return (p[..., :1] * c + p[..., 1:]).reshape(*c.shape[:-2], -1)


def _places(s):
    """(request, cache position) of each row, and its block and place in the block."""
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    pos = s["kv_len"].long()[seq] - (s["q_start"].long()[seq + 1] - row)
    return seq, pos, s["table"].long()[seq, pos // s["block"]], pos % s["block"]


# ---------------------------------------------------------------------------- inputs

def _batch(case, g):
    heads, kv_heads, dim = HEADS[case["model"]]
    q, n = _lens(case)
    block = case["block"]
    s = {"op": case["op"], "heads": heads, "kv_heads": kv_heads, "dim": dim, "group": case["group"], "block": block,
         "rows": int(q.sum()), "seqs": len(q), "max_q": int(q.max()), "max_len": int(n.max())}
    s["max_blocks"] = -(-s["max_len"] // block)
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(q)]).astype(np.int32)).cuda()
    s["kv_len"] = torch.from_numpy(n.astype(np.int32)).cuda()
    # blocks in pages of the pool (8 KB), scattered over it; a block nobody holds stays unused
    s["stride"] = -(-kv_heads * block * _token_bytes(dim, case["group"]) // 8192) * 8192
    held = torch.from_numpy(-(-n // block)).cuda()
    s["blocks"] = int(held.sum()) + 3
    order = torch.randperm(s["blocks"], generator=g, device="cuda").int()
    first = torch.cumsum(held, 0) - held
    j = torch.arange(s["max_blocks"], device="cuda")
    at = (first[:, None] + j[None, :]).clamp(max=s["blocks"] - 1)
    s["table"] = torch.where(j[None, :] < held[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
    s["cache"] = torch.full((s["blocks"] * s["stride"],), 255, dtype=torch.uint8, device="cuda")   # free places read as NaN
    return s


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "w4":
        s = {"op": "w4", "rows": case["rows"], "group": case["group"], "w": []}
        xs = {k: _normal(g, case["rows"], k).bfloat16() for k in sorted({k for _, k in PROJ[case["proj"]]})}
        for n, k in PROJ[case["proj"]]:
            c = (_normal(g, n, k) * 2.7 + 8).round().clamp(0, 15).to(torch.uint8)
            scales = (0.006 * (0.5 + torch.rand(k // case["group"], n, generator=g, device="cuda"))).half()
            zeros = None
            if case["zeros"]:
                z = torch.randint(5, 12, (k // case["group"], n), generator=g, device="cuda", dtype=torch.uint8)
                zeros = (z[:, 0::2] | (z[:, 1::2] << 4)).contiguous()
            s["w"].append({"x": xs[k], "codes": (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), "scales": scales, "zeros": zeros, "n": n, "k": k})
        return s
    s = _batch(case, g)
    heads, kv_heads, dim = s["heads"], s["kv_heads"], s["dim"]
    gain = 1.0 + 4.0 * (torch.rand(kv_heads * dim, generator=g, device="cuda") < 0.03)     # a few strong channels of the keys
    if case["op"] == "append":
        # one row of the fused projection's output: q, then k, then v
        s["qkv"] = _normal(g, s["rows"], (heads + 2 * kv_heads) * dim)
        s["qkv"][:, heads * dim:(heads + kv_heads) * dim] *= gain
        s["qkv"] = s["qkv"].bfloat16()
        s["pairs"] = case["pairs"]
        turn = torch.arange(s["max_len"], device="cuda")[:, None] * (10000.0 ** (-torch.arange(0, dim, 2, device="cuda") / dim))[None, :]
        s["cos"], s["sin"] = torch.cos(turn).contiguous(), torch.sin(turn).contiguous()
        return s
    # the cache as appends left it: every token that a request holds
    regions = _regions(s, s["cache"])
    n = s["kv_len"].long()
    for first in range(0, int(n.sum()), 1 << 16):
        t = torch.arange(first, min(first + (1 << 16), int(n.sum())), device="cuda")
        ends = torch.cumsum(n, 0)
        seq = torch.searchsorted(ends, t, right=True)
        pos = t - (ends - n)[seq]
        blk, at = s["table"].long()[seq, pos // s["block"]], pos % s["block"]
        for i in range(2):
            x = _normal(g, len(t), kv_heads, dim)
            codes, params = _quantise(x * gain.view(kv_heads, dim) if i == 0 else x, s["group"])
            regions[i][blk, :, at // 16, :, at % 16] = codes
            regions[2 + i][blk, :, at // 16, :, at % 16] = params
    s["q"] = _normal(g, s["rows"], heads * dim).bfloat16()
    s["scale"] = dim ** -0.5
    return s


# ---------------------------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, pairs):
    """x f32 [rows, heads, D] turned by the angles of its rows; pairs (2i, 2i + 1) or (i, i + D / 2)."""
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else x.chunk(2, -1)
    cos, sin = cos[:, None], sin[:, None]
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)


def _plain_append(s):
    heads, kv_heads, dim = s["heads"], s["kv_heads"], s["dim"]
    x = s["qkv"].float().view(s["rows"], -1, dim)
    _, pos, blk, at = _places(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _rotate(x[:, :heads], cos, sin, s["pairs"])
    k = _rotate(x[:, heads:heads + kv_heads], cos, sin, s["pairs"])
    regions = _regions(s, s["cache"])
    for i, y in enumerate((k, x[:, heads + kv_heads:])):
        codes, params = _quantise(y, s["group"])
        regions[i][blk, :, at // 16, :, at % 16] = codes
        regions[2 + i][blk, :, at // 16, :, at % 16] = params
    k, v = (_values(regions[i][blk, :, at // 16, :, at % 16], regions[2 + i][blk, :, at // 16, :, at % 16], s["group"]) for i in (0, 1))
    return {"q": q.bfloat16().flatten(1), "k": k.bfloat16().flatten(1), "v": v.bfloat16().flatten(1)}


def _plain_attend(s):
    heads, kv_heads, dim, seqs, most = s["heads"], s["kv_heads"], s["dim"], s["seqs"], s["max_q"]
    regions = _regions(s, s["cache"])
    table = s["table"].long().clamp(min=0)
    k, v = (_values(regions[i][table].movedim(4, 5), regions[2 + i][table].movedim(4, 5), s["group"])
            .movedim(2, 1).flatten(2, 4) for i in (0, 1))      # [seqs, kv heads, tokens, D]
    key = torch.arange(k.shape[2], device="cuda")
    held = key[None, :] < s["kv_len"][:, None]
    v = torch.where(held[:, None, :, None], v, 0.0)
    seq, pos, _, _ = _places(s)
    nth = torch.arange(s["rows"], device="cuda") - s["q_start"].long()[seq]
    q = torch.zeros(seqs, most, kv_heads, heads // kv_heads, dim, device="cuda")
    q[seq, nth] = s["q"].float().view(s["rows"], kv_heads, -1, dim)
    last = torch.full((seqs, most), -1, device="cuda")
    last[seq, nth] = pos
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                 # [seqs, kv heads, query heads x rows, D]
    a = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(seqs, kv_heads, -1, most, k.shape[2])
    a = torch.where((key <= last[..., None])[:, None, None], a, -torch.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top > -torch.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(seqs, kv_heads, -1, most, dim) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4)[seq, nth]                     # [rows, kv heads, query heads of one, D]
    return {"o": o.flatten(1).bfloat16(), "lse": lse.permute(0, 3, 1, 2)[seq, nth].flatten(1)}


def _plain_w4(s):
    out = []
    for w in s["w"]:
        c = torch.stack([w["codes"] & 15, w["codes"] >> 4], -1).view(w["n"], -1, s["group"]).float()
        z = 8.0
        if w["zeros"] is not None:
            z = torch.stack([w["zeros"] & 15, w["zeros"] >> 4], -1).flatten(1).t()[..., None].float()
        full = ((c - z) * w["scales"].float().t()[..., None]).flatten(1)
        out.append((w["x"].float() @ full.t()).bfloat16())
    return out


# ---------------------------------------------------------------------------- the library's calls

def _kept(s):
    """What a serving program makes once and keeps beside its buffers: descriptions, workspace, output buffers."""
    if "kept" in s:
        return s["kept"]
    import heterogeneous_adapters_gb300 as lora
    kept = {"lora": lora}
    if s["op"] == "w4":
        kept["y"] = [torch.empty(s["rows"], w["n"], dtype=torch.bfloat16, device="cuda") for w in s["w"]]
        kept["problems"] = lora.w4_problems([(w["x"], y, w["k"], w["n"], w["codes"], w["scales"], w["zeros"], w["n"], w["k"], s["group"])
                                             for w, y in zip(s["w"], kept["y"])])
        size = lora.w4_workspace_size(kept["problems"], s["rows"])
    else:
        kept["kv"] = lora.KvCache(s["cache"], s["blocks"], s["stride"], s["block"], s["kv_heads"], s["dim"], s["group"])
        kept["batch"] = lora.KvBatch(s["q_start"], s["kv_len"], s["table"], s["seqs"], s["rows"], s["max_blocks"], s["max_q"])
        empty = lambda heads: torch.empty(s["rows"], heads * s["dim"], dtype=torch.bfloat16, device="cuda")  # noqa: E731
        kept["q"], kept["k"], kept["v"] = empty(s["heads"]), empty(s["kv_heads"]), empty(s["kv_heads"])
        kept["lse"] = torch.empty(s["rows"], s["heads"], device="cuda")
        if s["op"] == "append":
            kept["rope"] = lora.Rope(s["cos"], s["sin"], s["max_len"], s["dim"], lora.LORA_ROPE_PAIRS if s["pairs"] else lora.LORA_ROPE_HALVES)
            a, b = s["heads"] * s["dim"], (s["heads"] + s["kv_heads"]) * s["dim"]
            kept["parts"] = s["qkv"][:, :a], s["qkv"][:, a:b], s["qkv"][:, b:]
        size = lora.kv_workspace_size(kept["kv"], kept["batch"], s["heads"])
    kept["size"], kept["ws"] = size, torch.empty(size, dtype=torch.uint8, device="cuda")
    lora.kv_workspace_init(kept["ws"], size, torch.cuda.current_stream().cuda_stream)
    s["kept"] = kept
    return kept


def _own(s):
    kept = _kept(s)
    lora, ws, size, stream = kept["lora"], kept["ws"], kept["size"], torch.cuda.current_stream().cuda_stream
    if s["op"] == "w4":
        lora.w4_matvec(kept["problems"], s["rows"], ws, size, stream)
        return kept["y"]
    if s["op"] == "append":
        q, k, v = kept["parts"]
        ld = s["qkv"].shape[1]
        lora.kv_append(kept["kv"], kept["batch"], q, ld, kept["q"], s["heads"] * s["dim"], s["heads"], k, ld, v, ld, kept["rope"], ws, size, stream)
        lora.kv_read(kept["kv"], kept["batch"], kept["k"], s["kv_heads"] * s["dim"], kept["v"], s["kv_heads"] * s["dim"], ws, size, stream)
        return {"q": kept["q"], "k": kept["k"], "v": kept["v"]}
    lora.kv_attend(kept["kv"], kept["batch"], s["q"], s["heads"] * s["dim"], s["heads"], s["scale"], kept["q"], s["heads"] * s["dim"],
                   kept["lse"], ws, size, stream)
    return {"o": kept["q"], "lse": kept["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "w4": _plain_w4}[state["op"]](state)


# ---------------------------------------------------------------------------- the definitions in 64 bits

def _exact_w4(s):
    out = []
    for w in s["w"]:
        low, high = (w["codes"] & 15).double(), (w["codes"] >> 4).double()
        full = torch.empty(w["n"], w["k"], dtype=torch.float64, device="cuda")
        full[:, 0::2], full[:, 1::2] = low, high
        for j in range(w["k"] // s["group"]):
            part = full[:, j * s["group"]:(j + 1) * s["group"]]
            zero = torch.full((w["n"],), 8.0, dtype=torch.float64, device="cuda")
            if w["zeros"] is not None:
                zero[0::2], zero[1::2] = (w["zeros"][j] & 15).double(), (w["zeros"][j] >> 4).double()
            part.sub_(zero[:, None]).mul_(w["scales"][j].double()[:, None])
        out.append(w["x"].double() @ full.T)
    return out


def _exact_append(s):
    heads, kv_heads, dim, group = s["heads"], s["kv_heads"], s["dim"], s["group"]
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    pos = torch.cat([torch.arange(n - (b - a), n) for a, b, n in zip(starts, starts[1:], lens)]).cuda()
    turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
    parts = list(s["qkv"].double().view(s["rows"], -1, dim).split([heads, kv_heads, kv_heads], 1))
    half = dim // 2
    for i in range(2):
        x = parts[i]
        if s["pairs"]:
            parts[i] = torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2)) * turn).reshape(x.shape)
        else:
            z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
            parts[i] = torch.cat([z.real, z.imag], -1)
    for i in (1, 2):
        x = parts[i].unflatten(-1, (dim // group, group))
        low = x.min(-1, keepdim=True).values
        step = ((x.max(-1, keepdim=True).values - low) / 15).half().double()
        middle = (low + 8 * step).half().double()
        parts[i] = (middle + step * torch.round((x - middle) / step).clamp(-8, 7)).flatten(-2)
    return {name: x.flatten(1) for name, x in zip("qkv", parts)}


def _exact_attend(s):
    heads, kv_heads, dim, group = s["heads"], s["kv_heads"], s["dim"], s["group"]
    tile = 16 * _token_bytes(dim, group)
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    cache = s["cache"].view(-1, s["stride"])[:, :kv_heads * s["block"] // 16 * tile].unflatten(1, (kv_heads, s["block"] // 16, tile))
    o = torch.zeros(s["rows"], heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["rows"], heads, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        used = cache[s["table"][i, :-(-n // s["block"])].long()]               # [blocks, kv heads, sub-tiles, bytes]
        rows = slice(starts[i], starts[i + 1])
        last = torch.arange(n - (starts[i + 1] - starts[i]), n, device="cuda")
        for h in range(kv_heads):
            mine = used[:, h].reshape(-1, tile)
            kv = []
            for part in range(2):
                b = mine[:, part * 8 * dim:(part + 1) * 8 * dim].view(-1, dim // 32, 16, 16)
                c = torch.empty(b.shape[0], 16, dim // 32, 32, dtype=torch.float64, device="cuda")
                c[..., 0::2], c[..., 1::2] = (b & 15).transpose(1, 2), (b >> 4).transpose(1, 2)
                at = 16 * dim + part * 64 * (dim // group)
                p = mine[:, at:at + 64 * (dim // group)].contiguous().view(torch.float16).view(-1, dim // group, 16, 2).double().transpose(1, 2)
                kv.append(((c.reshape(-1, 16, dim // group, group) - 8) * p[..., :1] + p[..., 1:]).reshape(-1, dim)[:n])
            mask = torch.arange(n, device="cuda")[None, :] > last[:, None]
            for j in range(h * (heads // kv_heads), (h + 1) * (heads // kv_heads)):
                a = s["q"][rows, j * dim:(j + 1) * dim].double() @ kv[0].T * s["scale"]
                a.masked_fill_(mask, -torch.inf)
                lse[rows, j] = torch.logsumexp(a, 1)
                o[rows, j] = torch.softmax(a, 1) @ kv[1]
    return {"o": o.flatten(1), "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "w4": _exact_w4}[case["op"]](s)
