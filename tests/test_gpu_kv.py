"""The 4-bit KV cache (include/lora_kv.h) against its definition in 64 bits: the append's
codes and rotation, the read-back, and the attention over the cache, at the shapes, lengths
and page layouts where they can go wrong."""
import numpy as np
import pytest

import heterogeneous_adapters_gb300 as lora

pytestmark = pytest.mark.gpu

KV, SEG = 0x40, 0x10


class Case:
    """A cache in scattered blocks with NaN bytes everywhere, and a batch over it."""

    def __init__(self, rows, lens, heads=8, kv_heads=2, dim=128, group=128, block=32, seed=0, pad=16, max_q=None):
        import torch
        self.torch, self.g = torch, torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.lens = list(rows), list(lens)
        self.heads, self.kv_heads, self.dim, self.group, self.block = heads, kv_heads, dim, group, block
        self.T, self.n = sum(rows), len(rows)
        self.bytes = lora.kv_block_bytes(block, kv_heads, dim, group)
        self.stride = self.bytes + pad
        held = [-(-max(n, 0) // block) for n in lens]
        self.blocks = sum(held) + 2
        self.max_blocks = max(held + [1])
        self.cache = torch.full((self.blocks * self.stride,), 255, dtype=torch.uint8, device="cuda")
        order = np.random.RandomState(seed).permutation(self.blocks)
        self.table_np = np.full((self.n, self.max_blocks), -1, np.int32)
        at = 0
        for i, h in enumerate(held):
            self.table_np[i, :h] = order[at:at + h]
            at += h
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
        self.q_start, self.kv_len, self.table = i32(np.concatenate([[0], np.cumsum(rows)])), i32(lens), i32(self.table_np)
        self.max_q = max_q if max_q is not None else max(self.rows + [0])
        self.kv = lora.KvCache(self.cache, self.blocks, self.stride, block, kv_heads, dim, group)
        self.batch = lora.KvBatch(self.q_start, self.kv_len, self.table, self.n, self.T, self.max_blocks, self.max_q)
        self.size = lora.kv_workspace_size(self.kv, self.batch, heads)
        self.ws = torch.empty(self.size, dtype=torch.uint8, device="cuda")
        self.stream = torch.cuda.current_stream().cuda_stream
        lora.kv_workspace_init(self.ws, self.size, self.stream)

    def normal(self, *shape, gain=1.0):
        return (self.torch.randn(*shape, generator=self.g, device="cuda") * gain).bfloat16()

    def error(self):
        return lora.get_device_error(self.ws, self.stream)

    # ---- the documented layout, in numpy
    def tiles(self):
        c = self.cache.cpu().numpy().reshape(self.blocks, self.stride)[:, :self.bytes]
        return c.reshape(self.blocks, self.kv_heads, self.block // 16, -1)

    def stored(self, seq, n):
        """K and V of tokens 0..n-1 of a request, fp64 [2][kv head][n][D]."""
        D, G = self.dim, self.group
        t = self.tiles()[self.table_np[seq, :-(-n // self.block)]]            # [blocks, heads, sub, bytes]
        t = np.moveaxis(t, 1, 0).reshape(self.kv_heads, -1, t.shape[-1])
        out = []
        for which in range(2):
            b = t[..., which * 8 * D:(which + 1) * 8 * D].reshape(self.kv_heads, -1, D // 32, 16, 16)
            c = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:4], 32).astype(np.float64)
            c = np.moveaxis(c, 2, 3).reshape(self.kv_heads, -1, D // G, G) - 8
            at = 16 * D + which * 64 * (D // G)
            p = np.ascontiguousarray(t[..., at:at + 64 * (D // G)]).view(np.float16).reshape(self.kv_heads, -1, D // G, 16, 2)
            p = np.moveaxis(p, 2, 3).reshape(self.kv_heads, -1, D // G, 2).astype(np.float64)
            out.append((c * p[..., :1] + p[..., 1:]).reshape(self.kv_heads, -1, D)[:, :n])
        return out

    # ---- calls
    def rope(self, rot=None, style=0, positions=None, max_pos=None, base=10000.0):
        rot = self.dim if rot is None else rot
        n = max_pos or max(max(self.lens), 1)
        if rot:
            a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)[None]
            self.cos = self.torch.tensor(np.cos(a), dtype=self.torch.float32, device="cuda")
            self.sin = self.torch.tensor(np.sin(a), dtype=self.torch.float32, device="cuda")
            return lora.Rope(self.cos, self.sin, n, rot, style, positions)
        return lora.Rope(None, None, 0, 0, style, positions)

    def append(self, q, k, v, rope, q_out=None):
        out = q_out if q_out is not None else self.torch.zeros(self.T, self.heads * self.dim, dtype=self.torch.bfloat16, device="cuda")
        lora.kv_append(self.kv, self.batch, q, q.stride(0), out, out.stride(0), self.heads, k, k.stride(0), v, v.stride(0),
                       rope, self.ws, self.size, self.stream)
        return out

    def read(self):
        k = self.torch.full((self.T, self.kv_heads * self.dim), 7.0, dtype=self.torch.bfloat16, device="cuda")
        v = k.clone()
        lora.kv_read(self.kv, self.batch, k, k.shape[1], v, v.shape[1], self.ws, self.size, self.stream)
        return k, v

    def attend(self, q, scale=None, lse=True):
        out = self.torch.full((self.T, self.heads * self.dim), 7.0, dtype=self.torch.bfloat16, device="cuda")
        ls = self.torch.full((self.T, self.heads), 7.0, device="cuda") if lse else None
        lora.kv_attend(self.kv, self.batch, q, q.stride(0), self.heads, scale or self.dim ** -0.5, out, out.shape[1], ls,
                       self.ws, self.size, self.stream)
        return out, ls

    def fill(self, gain=1.0, k=None):
        """Every token of every request appended (a call with all of them as rows), with random K or the given."""
        total = sum(max(n, 0) for n in self.lens)
        t = self.torch
        start = t.tensor(np.concatenate([[0], np.cumsum([max(n, 0) for n in self.lens])]), dtype=t.int32, device="cuda")
        lens = self.kv_len.clamp(min=0).int()
        batch = lora.KvBatch(start, lens, self.table, self.n, total, self.max_blocks, max(max(self.lens), 0))
        k = self.normal(total, self.kv_heads * self.dim, gain=gain) if k is None else k
        v = self.normal(total, self.kv_heads * self.dim)
        lora.kv_append(self.kv, batch, None, 0, None, 0, 0, k, k.shape[1], v, v.shape[1], self.rope(0), self.ws, self.size, self.stream)

    def check_attend(self, q, out, lse, scale=None):
        """Against softmax in 64 bits over the stored values.  The bounds: probabilities and
        outputs rounded to bf16 (2^-8 each, of sum p |v| and |o|);
        a score's fp32 sum over D terms is off by at most D 2^-24 sum |q k|."""
        scale = scale or self.dim ** -0.5
        q, out = q.double().cpu().numpy(), out.double().cpu().numpy()
        rep, row = self.heads // self.kv_heads, 0
        for s, (m, n) in enumerate(zip(self.rows, self.lens)):
            k, v = self.stored(s, max(n, 0)) if n > 0 else (np.zeros((self.kv_heads, 0, self.dim)),) * 2
            for i in range(m):
                last = n - m + i
                for h in range(self.heads):
                    got = out[row, h * self.dim:(h + 1) * self.dim]
                    if last < 0:
                        assert not got.any()
                        assert lse is None or float(lse[row, h]) == -np.inf
                        continue
                    kk, vv = k[h // rep, :last + 1], v[h // rep, :last + 1]
                    qq = q[row, h * self.dim:(h + 1) * self.dim]
                    a = scale * (kk @ qq)
                    top = a.max()
                    e = np.exp(a - top)
                    p = e / e.sum()
                    want = p @ vv
                    slack = float((scale * (np.abs(kk) @ np.abs(qq))).max()) * self.dim * 2.0 ** -24
                    tol = 2.0 ** -8 * (np.abs(want) + p @ np.abs(vv)) + slack * (p @ np.abs(vv)) + 1e-6
                    assert (np.abs(got - want) <= tol).all(), (s, i, h, np.abs(got - want).max())
                    if lse is not None:
                        w = top + np.log(e.sum())
                        assert abs(float(lse[row, h]) - w) <= slack + 2.0 ** -20 * (1 + abs(w)) + 1e-6, (s, i, h)
                row += 1


# ---------------------------------------------------------------------------- append and read

SHAPES = [dict(heads=8, kv_heads=2, dim=128, group=128, block=32), dict(heads=5, kv_heads=5, dim=128, group=32, block=16),
          dict(heads=6, kv_heads=3, dim=64, group=64, block=64), dict(heads=4, kv_heads=1, dim=64, group=32, block=48)]


def turned(x, cos, sin, rot, style):
    """x fp64 [rows, heads, D] turned by cos, sin fp64 [rows, rot / 2]."""
    y = x.copy()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if style else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, s = cos[:, None], sin[:, None]
    u, w = a * c - b * s, b * c + a * s
    if style:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, w
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = u, w
    return y


def check_append(case, q, k, v, q_out, pos, rot, style):
    D, G = case.dim, case.group
    to = lambda t, h: t.double().cpu().numpy().reshape(case.T, h, D)  # noqa: E731
    if rot:
        cos, sin = case.cos.double().cpu().numpy()[pos], case.sin.double().cpu().numpy()[pos]
    else:
        cos = sin = np.zeros((case.T, 0))
    turn = (lambda x: turned(x, cos, sin, rot, style)) if rot else (lambda x: x)
    wq = turn(to(q, case.heads))
    # fp32 rotation: two products and a sum, 3 roundings of values up to sqrt(2) |pair|; bf16 once (unit roundoff 2^-8)
    size = np.abs(to(q, case.heads)).max()
    assert (np.abs(to(q_out, case.heads) - wq) <= 2.0 ** -8 * np.abs(wq) + 2.0 ** -21 * size).all()
    rk, rv = (to(t, case.kv_heads) for t in case.read())
    for got, want in ((rk, turn(to(k, case.kv_heads))), (rv, to(v, case.kv_heads))):
        x = want.reshape(case.T, case.kv_heads, D // G, G)
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        step = (hi - lo) / 15
        # half a step, what rounding scale (15 steps of 2^-11) and offset to f16 shifts the ends
        # by, the subnormal step of f16, the fp32 rotation, and the bf16 of the read-back
        off = np.abs(lo) + 8 * step
        tol = 0.5 * step * (1 + 2.0 ** -10) + 2.0 ** -11 * (15 * step + off) + 16 * 2.0 ** -25
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -20 * (np.abs(lo) + np.abs(hi)) + 2.0 ** -8 * (np.abs(x) + step)
        err = np.abs(got.reshape(x.shape) - x)
        assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("rows,lens", [([1], [1]), ([1] * 5, [1, 16, 17, 100, 33]), ([7, 0, 40, 1], [7, 12, 130, 64]),
                                       ([130, 3], [200, 3])])
def test_append_and_read(cuda, shape, style, rows, lens):
    case = Case(rows, lens, seed=len(rows) + style, **shape)
    D = case.dim
    qkv = case.normal(case.T, (case.heads + 2 * case.kv_heads) * D + 8)
    q, k, v = qkv[:, :case.heads * D], qkv[:, case.heads * D:(case.heads + case.kv_heads) * D], qkv[:, (case.heads + case.kv_heads) * D:]
    v = v[:, :case.kv_heads * D]
    pos = np.concatenate([np.arange(n - m, n) for m, n in zip(rows, lens)])
    before = qkv.clone()
    out = case.append(q, k, v, case.rope(style=style))
    assert case.error() == 0
    check_append(case, q, k, v, out, pos, D, style)
    assert cuda.equal(qkv.view(cuda.int16), before.view(cuda.int16))
    # the second pass over the same rows leaves the same bytes
    bytes0 = case.cache.clone()
    out2 = case.append(q, k, v, case.rope(style=style))
    assert cuda.equal(bytes0, case.cache) and cuda.equal(out, out2)
    # only the rows' own places were written
    held = np.zeros((case.blocks, case.block), bool)
    for s, (m, n) in enumerate(zip(rows, lens)):
        for t in range(n - m, n):
            held[case.table_np[s, t // case.block], t % case.block] = True
    t = case.tiles()
    codes = t[..., :16 * D].reshape(case.blocks, case.kv_heads, case.block // 16, 2 * D // 32, 16, 16)
    codes = np.moveaxis(codes, 4, 3).reshape(case.blocks, case.kv_heads, case.block, -1)
    assert (np.moveaxis(codes, 1, 2)[~held] == 255).all()
    assert (case.cache.cpu().numpy().reshape(case.blocks, case.stride)[:, case.bytes:] == 255).all()


def test_append_partial_rotation_given_positions_and_in_place(cuda):
    case = Case([3, 2], [40, 9], heads=4, kv_heads=2, dim=128, group=32, block=16)
    q, k, v = case.normal(5, 512), case.normal(5, 256), case.normal(5, 256)
    pos = np.array([5, 0, 77, 3, 3])
    rope = case.rope(rot=48, style=0, positions=cuda.tensor(pos, dtype=cuda.int32, device="cuda"), max_pos=78)
    qin = q.clone()
    out = case.append(q, k, v, rope, q_out=q)
    assert case.error() == 0
    check_append(case, qin, k, v, out, pos, 48, 0)
    case = Case([3, 2], [40, 9], heads=4, kv_heads=2, dim=128, group=128, block=16)
    out = case.append(qin, k, v, case.rope(0))
    check_append(case, qin, k, v, out, None, 0, 0)


def test_append_values_at_the_ends_of_the_range(cuda):
    """Constant groups, tiny and huge values, a group with an infinity or a NaN."""
    case = Case([6], [6], heads=2, kv_heads=1, dim=64, group=32, block=16)
    k = case.normal(6, 64)
    k[0] = 3.0
    k[1] *= 1e-9
    k[2] = k[2] * 1e30
    k[3, 5] = float("inf")
    k[4, 40] = float("nan")
    k[5, :32] = 0.0
    q, v = case.normal(6, 128), case.normal(6, 64)
    case.append(q, k, v, case.rope(0))
    rk, rv = case.read()
    rk = rk.float().cpu().numpy()
    assert (rk[0] == 3.0).all() and (rk[5, :32] == 0).all()
    assert np.abs(rk[1]).max() <= 1e-7                      # below f16's smallest step
    assert np.isfinite(rk[2]).all() and np.abs(rk[2]).max() <= 16 * 65504
    assert np.isnan(rk[3, :32]).all() and np.isfinite(rk[3, 32:]).all()
    assert np.isnan(rk[4, 32:]).all() and np.isfinite(rk[4, :32]).all()
    assert case.error() == 0


# ---------------------------------------------------------------------------- attention

@pytest.mark.parametrize("shape", SHAPES + [dict(heads=32, kv_heads=2, dim=128, group=128, block=16),
                                            dict(heads=24, kv_heads=1, dim=64, group=64, block=128)])
@pytest.mark.parametrize("rows,lens", [([1], [1]), ([1], [1000]), ([1] * 6, [15, 16, 17, 64, 65, 300]),
                                       ([2, 0, 5, 1, 3], [2, 50, 129, 31, 64]), ([70, 1], [100, 200])])
def test_attend(cuda, shape, rows, lens):
    case = Case(rows, lens, seed=3, **shape)
    case.fill()
    q = case.normal(case.T, case.heads * case.dim)
    out, lse = case.attend(q)
    assert case.error() == 0
    case.check_attend(q, out, lse)
    again, lse2 = case.attend(q)
    assert cuda.equal(out.view(cuda.int16), again.view(cuda.int16)) and cuda.equal(lse, lse2)
    third, _ = case.attend(q, lse=False)
    assert cuda.equal(out.view(cuda.int16), third.view(cuda.int16))


def test_attend_rows_without_tokens_and_empty_requests(cuda):
    """Requests shorter than their rows (the first rows see nothing), of length zero, without rows."""
    case = Case([3, 1, 0, 2, 1], [1, 0, 40, 2, 33], heads=4, kv_heads=2, block=16)
    case.fill()
    q = case.normal(case.T, 512)
    out, lse = case.attend(q)
    assert case.error() == 0
    case.check_attend(q, out, lse)


@pytest.mark.parametrize("gain,scale", [(40.0, 1.0), (1e-3, 1.0), (8.0, 0.01)])
def test_attend_peaked_and_flat_scores(cuda, gain, scale):
    case = Case([1, 4], [777, 200], heads=8, kv_heads=2)
    case.fill(gain=gain)
    q = case.normal(case.T, 8 * 128)
    out, lse = case.attend(q, scale=scale)
    case.check_attend(q, out, lse, scale=scale)


def test_attend_long_context_and_strided_rows(cuda):
    """A context split over many workers, q and out as slices of wider rows."""
    case = Case([1, 1, 2], [20011, 7, 4096], heads=8, kv_heads=2, block=64, seed=5)
    case.fill()
    wide = case.normal(case.T, 8 * 128 + 24)
    q = wide[:, 8:8 + 8 * 128]
    out, lse = case.attend(q)
    assert case.error() == 0
    case.check_attend(q.contiguous(), out, lse)


def test_attend_chunk_of_a_prompt(cuda):
    """Many rows of one request, next to single-token requests in the same call."""
    case = Case([150, 1, 37, 1], [290, 500, 37, 3], heads=8, kv_heads=2, block=32, seed=6)
    case.fill()
    q = case.normal(case.T, 8 * 128)
    out, lse = case.attend(q)
    assert case.error() == 0
    case.check_attend(q, out, lse)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("which", [0, 2])
def test_attend_chunk_where_some_rows_rise_with_every_block(cuda, dim, which):
    """Eight rows' scores rise by 8 with every 128 tokens and the others' stay: rows that take a
    new reference at every block beside rows that never do."""
    case = Case([32, 24], [2048, 1500], heads=8, kv_heads=2, dim=dim, group=dim, block=32, seed=8)
    d = cuda.where(cuda.arange(dim, device="cuda") % 2 == 0, 1.0, -1.0) * dim ** -0.5
    at = cuda.cat([cuda.arange(n, device="cuda") for n in case.lens]) // 128
    k = case.normal(sum(case.lens), 2, dim, gain=0.5).float() + (at * 8.0)[:, None, None] * d * dim ** 0.5 / 32.0
    case.fill(k=k.bfloat16().reshape(-1, 2 * dim))
    q = case.normal(case.T, 8, dim).float()
    for first in (0, 32):
        rows = slice(first + 8 * which, first + 8 * which + 8)
        q[rows] = 32.0 * d + 0.25 * q[rows]
    q = q.bfloat16().reshape(case.T, 8 * dim)
    out, lse = case.attend(q)
    assert case.error() == 0
    case.check_attend(q, out, lse)


def test_attend_block_in_offsets_beyond_32_bits(cuda):
    """A block that starts more than 4 GB after the first."""
    case = Case([1, 2], [100, 50], heads=4, kv_heads=2, block=32)
    far = -(-(1 << 32) // case.stride) + 3
    big = cuda.empty((far + case.blocks) * case.stride, dtype=cuda.uint8, device="cuda")
    big[far * case.stride:] = 255
    case.cache = big[far * case.stride:]
    case.kv = lora.KvCache(big, far + case.blocks, case.stride, 32, 2, 128, 128)
    small = case.table.clone()
    case.table += cuda.where(small >= 0, far, 0).int()
    case.fill()
    q = case.normal(case.T, 512)
    out, lse = case.attend(q)
    assert case.error() == 0
    case.check_attend(q, out, lse)


def test_append_then_attend_as_a_decode_loop(cuda):
    """Tokens appended one step at a time, across block ends, on a stream of its own."""
    case = Case([1, 1], [70, 35], heads=4, kv_heads=2, block=16)
    side = cuda.cuda.Stream()
    side.wait_stream(cuda.cuda.current_stream())
    case.stream = side.cuda_stream
    with cuda.cuda.stream(side):
        for step in range(70):
            lens = np.array([step + 1, max(0, step - 34)])
            case.kv_len.copy_(cuda.tensor(lens, dtype=cuda.int32))
            q, k, v = case.normal(2, 512), case.normal(2, 256), case.normal(2, 256)
            out_q = case.append(q, k, v, case.rope(style=1, max_pos=80))
            if step in (0, 15, 16, 40, 69):
                out, lse = case.attend(out_q)
                case.lens = [int(n) for n in lens]
                case.check_attend(out_q, out, lse)
    assert case.error() == 0


# ---------------------------------------------------------------------------- data errors

def bad_case():
    """Requests of 2, 1 and 1 rows over 40, 20 and 5 tokens, and what they give."""
    case = Case([2, 1, 1], [40, 20, 5], heads=4, kv_heads=2, block=16)
    case.fill()
    case.x = case.normal(4, 512), case.normal(4, 256), case.normal(4, 256)
    case.good, _ = case.attend(case.x[0])
    assert case.error() == 0
    return case


@pytest.mark.parametrize("bad", ["id", "negative", "long"])
def test_bad_blocks_set_the_bit_and_spare_other_requests(cuda, bad):
    case = bad_case()
    if bad == "long":
        case.kv_len[0] = 16 * case.max_blocks + 3
    else:
        case.table[0, 2 if bad == "id" else 0] = case.blocks if bad == "id" else -7
    out, _ = case.attend(case.x[0])
    assert case.error() == KV
    # (how the work is split, and with it the last bit, may change with a request's length)
    assert bool((out[2:].float() - case.good[2:].float()).abs().max() <= 2.0 ** -6)
    assert not cuda.equal(out[:2], case.good[:2])
    # (a request that claims tokens nobody appended reads whatever its blocks hold)
    assert bad == "long" or bool(out.isfinite().all())
    case.kv_len[0] = 34                                    # both rows in block 2
    if bad == "long":
        case.kv_len[0] = 16 * case.max_blocks + 2
    if bad == "negative":
        case.table[0, 2] = -7
    before = case.cache.clone()
    case.append(*case.x, case.rope(0))
    assert case.error() == KV
    case.table[1:] = -1
    case.kv_len[1:] = 0
    after = case.cache.clone()
    case.append(*case.x, case.rope(0))                     # the bad request alone: nothing is written
    assert case.error() == KV and cuda.equal(after, case.cache) and not cuda.equal(before, after)


def test_bad_rows_and_positions_set_their_bits(cuda):
    case = bad_case()
    case.batch = lora.KvBatch(case.q_start, case.kv_len, case.table, 3, 4, case.max_blocks, 1)
    out, _ = case.attend(case.x[0])                        # request 0 has more rows than promised
    assert case.error() == KV and bool((out[:2] == 7).all())
    assert bool((out[2:].float() - case.good[2:].float()).abs().max() <= 2.0 ** -6)
    for start in ([0, 9, 3, 4], [0, 2, 1, 4], [-1, 2, 3, 4], [0, 2, 3, 9]):
        case = bad_case()
        case.q_start.copy_(cuda.tensor(start, dtype=cuda.int32))
        case.batch = lora.KvBatch(case.q_start, case.kv_len, case.table, 3, 4, case.max_blocks, 16)
        case.attend(case.x[0])
        assert case.error() & SEG, start
        case.append(*case.x, case.rope(0))
        assert case.error() & SEG, start
    case = bad_case()
    before = case.cache.clone()
    out = case.append(*case.x, case.rope(max_pos=4))       # tokens 38, 39, 19 and 4
    assert case.error() == KV and cuda.equal(before, case.cache) and not bool(out.any())


def test_refusals(cuda):
    from heterogeneous_adapters_gb300 import _binding as B
    case = bad_case()
    q, k, v = case.x
    out, z = cuda.zeros_like(q), (case.ws, case.size, case.stream)

    def status(f, *a):
        with pytest.raises(lora.LoraError) as e:
            f(*a)
        return e.value.status

    odd = cuda.zeros(4, 520, dtype=cuda.bfloat16, device="cuda")
    assert status(lora.kv_attend, case.kv, case.batch, q, 512, 3, 0.1, out, 512, None, *z) == B.LORA_EINVAL
    assert status(lora.kv_attend, case.kv, case.batch, q, 512, 4, float("nan"), out, 512, None, *z) == B.LORA_EINVAL
    assert status(lora.kv_attend, case.kv, case.batch, q, 504, 4, 0.1, out, 512, None, *z) == B.LORA_EINVAL
    assert status(lora.kv_attend, case.kv, case.batch, odd[:, 1:], 520, 4, 0.1, out, 512, None, *z) == B.LORA_EALIGN
    assert status(lora.kv_attend, case.kv, case.batch, q, 513, 4, 0.1, out, 512, None, *z) == B.LORA_EALIGN
    assert status(lora.kv_attend, case.kv, case.batch, q, 512, 4, 0.1, None, 512, None, *z) == B.LORA_EINVAL
    assert status(lora.kv_attend, case.kv, case.batch, q, 512, 4, 0.1, out, 512, None, case.ws, 0, case.stream) == B.LORA_EWORKSPACE
    assert status(lora.kv_append, case.kv, case.batch, q, 512, out, 512, 4, k, 248, v, 256, case.rope(0), *z) == B.LORA_EINVAL
    assert status(lora.kv_append, case.kv, case.batch, q, 512, out, 512, 4, k, 256, v, 256, lora.Rope(None, None, 5, 64), *z) == B.LORA_EINVAL
    assert status(lora.kv_append, case.kv, case.batch, q, 512, out, 512, 4, k, 256, v, 256, case.rope(24), *z) == B.LORA_EINVAL
    assert status(lora.kv_read, case.kv, case.batch, k, 256, None, 256, *z) == B.LORA_EINVAL
    small = lora.KvCache(case.cache, case.blocks, case.bytes - 16, 16, 2, 128, 128)
    assert status(lora.kv_attend, small, case.batch, q, 512, 4, 0.1, out, 512, None, *z) == B.LORA_EINVAL
    assert case.error() == 0
    # nothing to do
    none = lora.KvBatch(case.q_start, case.kv_len, case.table, 0, 0, case.max_blocks, 0)
    lora.kv_attend(case.kv, none, q, 512, 4, 0.1, out, 512, None, *z)
    assert not bool(out.any())
