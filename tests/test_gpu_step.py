"""The decode step of examples/decode_step.py: each stage against its definition in 64 bits on
the values the stage before left."""
import os
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def product(torch, layer, i, x):
    """x W^T + the requests' deltas, fp64, and the size of the sums."""
    codes, scales, zeros = layer.weights[i]
    k, n = layer.dims[i]
    G, r = layer.weight_group, layer.rank
    c = torch.stack([codes & 15, codes >> 4], -1).view(n, k // G, G).double()
    z = torch.stack([zeros & 15, zeros >> 4], -1).view(k // G, n).t()[..., None].double()
    w = ((c - z) * scales.t()[..., None].double()).view(n, k)
    x = x.double()
    y, size = x @ w.t(), x.abs() @ w.abs().t()
    pages = lambda d: -(-d // layer.h)  # noqa: E731
    pre = sum(pages(a) + pages(b) for a, b in layer.dims[:i])
    for t, a in enumerate(layer.adapter.tolist()):
        if a < 0:
            continue
        at = int(layer.pt_off[a]) + r * pre
        ids = layer.page_table[at:at + r * (pages(k) + pages(n))].long()
        rows = layer.pages[ids].double()
        A = rows[:r * pages(k)].view(pages(k), r, -1).transpose(0, 1).reshape(r, -1)[:, :k]
        B = rows[r * pages(k):].view(pages(n), r, -1).transpose(0, 1).reshape(r, -1)[:, :n]
        d = (x[t] @ A.t()) * 2.0
        y[t] += d @ B
        size[t] += (x[t].abs() @ A.abs().t()) * 2.0 @ B.abs()
    return y, size


def near(got, want, size):
    """Two roundings to bf16 (the base product and the sum with the delta, 2^-8 each) and fp32 sums."""
    return bool(((got.double() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -7 * 2.0 ** -3 * size).all())


@pytest.mark.parametrize("shape", [dict(h=512, heads=8, kv_heads=2, dim=128, kv_group=128, block=32),
                                   dict(h=1024, heads=6, kv_heads=3, dim=64, kv_group=32, block=16)])
def test_decode_steps(cuda, shape):
    from decode_step import Layer
    torch = cuda
    layer = Layer(requests=5, max_len=64, adapters=3, rank=8, weight_group=64, **shape)
    nq = layer.heads * layer.dim
    hist = [[], []]
    for step in range(20):
        x = torch.randn(layer.T, layer.h, device="cuda").bfloat16()
        out = layer.step(x)
        assert layer.errors() == 0
        for i, y in enumerate(layer.parts):
            want, size = product(torch, layer, i, x)
            assert near(y, want, size), i
        # attention over every token so far as the cache holds it (read back as the batch of all tokens)
        import heterogeneous_adapters_gb300 as lora
        n = step + 1
        start = (torch.arange(layer.T + 1, device="cuda") * n).int()
        every = lora.KvBatch(start, layer.kv_len, layer.table, layer.T, layer.T * n, layer.max_blocks, n)
        k = torch.empty(layer.T * n, layer.kv_heads * layer.dim, dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        stream = torch.cuda.current_stream().cuda_stream
        lora.kv_read(layer.kv, every, k, k.shape[1], v, v.shape[1], layer.step_ws, layer.step_bytes, stream)
        # this step's keys and values are within half a step of 15 (and bf16) of what was projected
        proj_v = layer.parts[2].double().view(layer.T, -1, layer.kv_group)
        held = v.view(layer.T, n, -1)[:, -1].double().view(layer.T, -1, layer.kv_group)
        span = proj_v.amax(-1, keepdim=True) - proj_v.amin(-1, keepdim=True)
        assert bool(((held - proj_v).abs() <= span / 30 * 1.01 + 2.0 ** -8 * (proj_v.abs() + span)).all())
        hist[0].append(k), hist[1].append(v)
        rep = layer.heads // layer.kv_heads
        kk = k.double().view(layer.T, n, layer.kv_heads, layer.dim).repeat_interleave(rep, 2)
        vv = v.double().view(layer.T, n, layer.kv_heads, layer.dim).repeat_interleave(rep, 2)
        q = layer.q.double().view(layer.T, layer.heads, layer.dim)
        a = torch.einsum("thd,tnhd->thn", q, kk) * layer.dim ** -0.5
        p = torch.softmax(a, -1)
        want = torch.einsum("thn,tnhd->thd", p, vv).flatten(1)
        # the read-back rounds keys and values to bf16: scores off by 2^-8 sum |q k|
        shift = (2.0 ** -8 * torch.einsum("thd,tnhd->thn", q.abs(), kk.abs()) * layer.dim ** -0.5).amax(-1)
        size = torch.einsum("thn,tnhd->thd", p, vv.abs())
        tol = (2.0 ** -6 + 2 * shift[..., None]) * size
        assert bool(((layer.att.double() - want).abs() <= tol.flatten(1) + 1e-6).all())
        want, size = product(torch, layer, 3, layer.att)
        assert near(out, want, size)
