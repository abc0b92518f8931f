"""Attention over a 4-bit cache in 64 bits, on the GPU, and the bounds that include/lora_kv.h
gives for the kernels' results."""
import torch


def tokens(case, seq, n):
    """Tokens 0 .. n - 1 of a request as the cache holds them: for K and V (scale (c - 8), offset),
    each fp64 [kv head][n][D], whose sum is the value."""
    D, G, heads = case.dim, case.group, case.kv_heads
    blocks = case.table[seq, :-(-n // case.block)].long().clamp(min=0)
    t = case.cache.view(case.blocks, case.stride)[:, :case.bytes][blocks]
    t = t.view(len(blocks), heads, case.block // 16, -1).transpose(0, 1).reshape(heads, -1, case.bytes // (heads * case.block // 16))
    out = []
    for which in range(2):
        b = t[..., which * 8 * D:(which + 1) * 8 * D].reshape(heads, -1, D // 32, 16, 16)
        c = torch.stack([b & 15, b >> 4], -1).reshape(heads, -1, D // 32, 16, 32).transpose(2, 3).reshape(heads, -1, D // G, G)[:, :n]
        at = 16 * D + which * 64 * (D // G)
        p = t[..., at:at + 64 * (D // G)].contiguous().view(torch.float16).view(heads, -1, D // G, 16, 2)
        p = p.transpose(2, 3).reshape(heads, -1, D // G, 2)[:, :n].double()
        out.append((((c.double() - 8) * p[..., :1]).flatten(2), p[..., 1:].expand(-1, -1, -1, G).flatten(2)))
    return out


def check(case, q, out, lse, scale=None, heads=None):
    """Every visible token counts (one whose block is missing is not there), in 64 bits over the stored values, with
      - 2^-8 of the result: bf16;
      - 2^-10 of sum p |v|: the weight rounds to f16 (2^-11 of itself), and so does v over its
        power of two, or a scale below 2^-14 of its offset stands as that (2^-11 of v);
      - fp32 sums: scores off by D 2^-24 of the sums of their parts, outputs by 2^-14;
      - per token 2^-29 of the row's largest p (scale |c - 8| + |offset|): weights that small are
        multiples of f16's smallest step.
    A token whose V is not a number makes its group of the output one, and nothing else."""
    scale = scale or case.dim ** -0.5
    rep, row = case.heads // case.kv_heads, 0
    for s, (m, n) in enumerate(zip(case.rows, case.lens)):
        (kc, ko), (vc, vo) = tokens(case, s, n)
        first = torch.arange(n - m, n, device="cuda")
        token = torch.arange(n, device="cuda")
        hide = (token[None] > first[:, None]) | (case.table[s, token // case.block] < 0)[None]
        for h in heads if heads is not None else range(case.heads):
            a, o = (kc[h // rep], ko[h // rep])
            qq = q[row:row + m].double()[:, h * case.dim:(h + 1) * case.dim]
            z = (qq @ (a + o).t() * scale).masked_fill(hide, -torch.inf)
            size = (qq.abs() @ (a.abs() + o.abs()).t() * scale).masked_fill(hide, 0).amax(1, keepdim=True)
            slack = size * case.dim * 2.0 ** -24
            want_lse = torch.logsumexp(z, 1, keepdim=True)
            p = torch.exp(z - want_lse)
            a, o = vc[h // rep], vo[h // rep]
            v, parts = a + o, a.abs() + o.abs()
            gone = v.isnan()
            lost = (p * (~hide)) @ gone.double() > 0              # groups that a token makes NaN
            v, parts = v.nan_to_num(0.0), parts.nan_to_num(0.0)
            want, weight = p @ v, p @ v.abs()
            step = (p * parts.amax(-1)).amax(1, keepdim=True)
            got = out[row:row + m, h * case.dim:(h + 1) * case.dim].double()
            tol = (2.0 ** -8 * want.abs() + 2.0 ** -10 * weight + (2 * slack + 2.0 ** -14) * (p @ parts)
                   + n * 2.0 ** -29 * step + 1e-9)
            assert bool((got.isnan() == lost).all()), (s, h, int(got.isnan().sum()), int(lost.sum()))
            err = ((got - want).abs() - tol).masked_fill(lost, -1.0)
            assert bool((err <= 0).all()), (s, h, float(err.max()), float((got - want).abs().masked_fill(lost, 0).max()))
            off = (lse[row:row + m, h:h + 1].double() - want_lse).abs()
            assert bool((off <= slack + 2.0 ** -17 * (1 + want_lse.abs())).all()), (s, h, float(off.max()))
        row += m
