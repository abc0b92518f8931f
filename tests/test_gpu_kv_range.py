"""Attention over the 4-bit cache where the weights of tokens differ by many powers of two, where a
visible token is not a number, and at the ends of the arguments' ranges; against 64 bits with the
bounds of tests/kv_exact.py."""
import numpy as np
import pytest

import heterogeneous_adapters_gb300 as lora

from .kv_exact import check
from .test_gpu_kv import SEG, Case

pytestmark = pytest.mark.gpu

FORMS = [(64, 64), (64, 32), (128, 128), (128, 32)]


def fill(case, k, v):
    """Every token of every request: k, v [tokens][kv heads * D], appended as they are."""
    t = case.torch
    start = t.tensor(np.concatenate([[0], np.cumsum(case.lens)]), dtype=t.int32, device="cuda")
    total = sum(case.lens)
    batch = lora.KvBatch(start, case.kv_len, case.table, case.n, total, case.max_blocks, max(case.lens))
    lora.kv_append(case.kv, batch, None, 0, None, 0, 0, k, k.shape[1], v, v.shape[1], case.rope(0), case.ws, case.size, case.stream)


def signs(torch, dim, every=1):
    return torch.where(torch.arange(dim, device="cuda") // every % 2 == 0, 1.0, -1.0)


# ---------------------------------------------------------------------------- tokens that are not numbers

@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("n", [64, 70, 95, 96, 300])
@pytest.mark.parametrize("back", [1, 2, 20, 60])
def test_a_visible_token_that_is_not_a_number_shows(cuda, dim, group, rows, n, back):
    """V of one token, `back` from the end, holds a NaN: the rows that see it are NaN in its group of
    V, the rows before it and the other groups are as without it."""
    case = Case([rows], [max(n, rows)], heads=4, kv_heads=2, dim=dim, group=group, block=16, seed=n)
    k, v = case.normal(case.lens[0], 2 * dim), case.normal(case.lens[0], 2 * dim)
    v[case.lens[0] - back, dim + 5] = float("nan")
    fill(case, k, v)
    q = case.normal(rows, 4 * dim)
    out, lse = case.attend(q)
    assert case.error() == 0
    assert bool(out.isnan().any()) and not bool(out[:, :2 * dim].isnan().any())
    check(case, q, out, lse)


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("back", [1, 20, 200, 290])
@pytest.mark.parametrize("gap", [-300.0, 300.0])
def test_a_token_that_is_not_a_number_at_any_weight(cuda, dim, group, rows, back, gap):
    """The same where the token's weight is 2^gap of the others', beyond what fp32 holds."""
    case = Case([rows], [300], heads=4, kv_heads=2, dim=dim, group=group, block=16, seed=5)
    s = signs(cuda, dim)
    k = cuda.zeros(300, 2, dim, device="cuda")
    k[300 - back] = gap * np.log(2.0) * dim ** -0.5 * s
    v = case.normal(300, 2 * dim)
    v[300 - back, dim + 5] = float("nan")
    fill(case, k.flatten(1).bfloat16(), v)
    q = s.repeat(rows, 4).bfloat16()
    out, lse = case.attend(q)
    assert case.error() == 0
    check(case, q, out, lse)


# ---------------------------------------------------------------------------- weights far apart

GAPS = [-4.0, 4.0, 6.0, 7.0, 8.0, 10.0, 12.0, 12.7, 13.0, 15.0, 20.0, 24.0]


def flat_beside_wide(torch, rows, n, kv_heads, repeats, dim, group, wide, flat):
    """Tokens whose V is (nearly) constant beside one whose V is wide, at distances of their scores
    from -4 to 24 powers of two: the many flat ones keep their share."""
    gaps = GAPS * repeats
    case = Case([rows] * len(gaps), [n - i % 12 for i in range(len(gaps))], heads=4 * kv_heads, kv_heads=kv_heads, dim=dim, group=group,
                block=64, seed=1)
    s, at, ks, vs = signs(torch, dim), n // 4, [], []
    for gap, n in zip(gaps, case.lens):
        k = torch.zeros(n, kv_heads, dim, device="cuda")
        k[at] = gap * np.log(2.0) * dim ** -0.5 * s
        noise = torch.randn(n, kv_heads, dim, generator=case.g, device="cuda")
        v = {"constant": torch.ones_like(noise), "near": 1 + 2.0 ** -7 * noise, "offset": 3 + 0.25 * noise}[flat]
        v[at] = wide * signs(torch, dim, 3)
        ks.append(k.flatten(1)), vs.append(v.flatten(1))
    fill(case, torch.cat(ks).bfloat16(), torch.cat(vs).bfloat16())
    q = s.repeat(case.T, 4 * kv_heads).bfloat16()
    out, lse = case.attend(q)
    assert case.error() == 0
    check(case, q, out, lse, heads=[0, 4 * kv_heads - 1])


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("wide", [2.6, 120.0])
@pytest.mark.parametrize("flat", ["constant", "near", "offset"])
@pytest.mark.parametrize("rows,n,kv_heads,repeats", [(1, 4096, 1, 1), (1, 300, 8, 16), (3, 150, 8, 16)])
def test_flat_tokens_beside_a_wide_one_few_rows(cuda, dim, group, wide, flat, rows, n, kv_heads, repeats):
    flat_beside_wide(cuda, rows, n, kv_heads, repeats, dim, group, wide, flat)


@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("wide", [2.6, 120.0])
@pytest.mark.parametrize("flat", ["constant", "near", "offset"])
def test_flat_tokens_beside_a_wide_one_many_rows(cuda, dim, group, wide, flat):
    flat_beside_wide(cuda, 16, 4096, 1, 1, dim, group, wide, flat)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 16])
def test_groups_of_different_sizes(cuda, dim, rows):
    """Groups of one head whose V differs in size by 2^16: the small ones are exact too."""
    case = Case([rows, 1], [700, 333], heads=4, kv_heads=2, dim=dim, group=32, block=32, seed=2)
    total = sum(case.lens)
    size = 2.0 ** (cuda.arange(2 * dim, device="cuda") // 32 % (dim // 32) * -(16 // (dim // 32 - 1))).float()
    v = case.normal(total, 2 * dim).float() * 64.0 * size
    fill(case, case.normal(total, 2 * dim, gain=1.5), v.bfloat16())
    q = case.normal(case.T, 4 * dim)
    out, lse = case.attend(q)
    assert case.error() == 0
    check(case, q, out, lse)


# ---------------------------------------------------------------------------- ordinary values, tightly

@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("rows,lens", [([1], [33]), ([1, 1, 1], [1000, 31, 4097]), ([3, 1, 5], [129, 2000, 64]), ([150, 1, 20], [900, 50, 20])])
def test_ordinary_values(cuda, dim, group, rows, lens):
    case = Case(rows, lens, heads=8, kv_heads=2, dim=dim, group=group, block=48, seed=3)
    total = sum(lens)
    fill(case, case.normal(total, 2 * dim), case.normal(total, 2 * dim))
    q = case.normal(case.T, 8 * dim)
    out, lse = case.attend(q)
    assert case.error() == 0
    check(case, q, out, lse)


# ---------------------------------------------------------------------------- the ends of the arguments

@pytest.mark.parametrize("dim,group", FORMS)
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 3e38])
@pytest.mark.parametrize("rows", [1, 20])
def test_zero_queries_at_any_scale(cuda, dim, group, scale, rows):
    """q = 0: the mean of the visible values, whatever the scale."""
    case = Case([rows, 2], [77, 40], heads=4, kv_heads=1, dim=dim, group=group, block=16, seed=4)
    total = sum(case.lens)
    fill(case, case.normal(total, dim), case.normal(total, dim))
    q = cuda.zeros(case.T, 4 * dim, dtype=cuda.bfloat16, device="cuda")
    out, lse = case.attend(q, scale=scale)
    assert case.error() == 0
    check(case, q, out, lse, scale=scale)


@pytest.mark.parametrize("length", [-5, -(1 << 31)])
def test_negative_lengths_hold_no_token(cuda, length):
    """As any length below the request's rows: nothing appended, zeros read back and attended, no error."""
    case = Case([1, 2, 60], [20, 30, 80], heads=4, kv_heads=2, dim=128, group=128, block=16)
    case.fill()
    q, k, v = case.normal(63, 512), case.normal(63, 256), case.normal(63, 256)
    case.kv_len.copy_(cuda.tensor([20, length, length], dtype=cuda.int32))
    before = case.cache.clone()
    out = case.append(q, k, v, case.rope())
    rk, rv = case.read()
    o, lse = case.attend(q)
    assert case.error() == 0
    assert not bool(out[1:].any()) and not bool(rk[1:].any()) and not bool(rv[1:].any()) and not bool(o[1:].any())
    assert bool((lse[1:] == -float("inf")).all()) and bool(o[0].any())
    case.kv_len[0] = length
    case.cache.copy_(before)
    case.append(q, k, v, case.rope())
    assert case.error() == 0 and cuda.equal(before, case.cache)


@pytest.mark.parametrize("start", [[0, 2, 4, 9], [-3, -1, 2, 4], [0, 1, 5, 5]])
def test_every_call_reports_rows_outside_the_batch(cuda, start):
    """Requests whose rows leave [0, T] set the segment bit, also where none of their rows is a row of the batch."""
    case = Case([2, 1, 1], [40, 20, 5], heads=4, kv_heads=2, block=16)
    case.fill()
    assert case.error() == 0
    case.q_start.copy_(cuda.tensor(start, dtype=cuda.int32))
    case.batch = lora.KvBatch(case.q_start, case.kv_len, case.table, 3, 4, case.max_blocks, 16)
    q, k, v = case.normal(4, 512), case.normal(4, 256), case.normal(4, 256)
    for call in (lambda: case.append(q, k, v, case.rope()), case.read, lambda: case.attend(q)):
        call()
        assert case.error() == SEG


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("requests", [4, 40])
def test_requests_of_either_kernel_in_one_call(cuda, dim, requests):
    """Requests of 28 to 56 packed rows, on both sides of where the kernel for many rows takes over."""
    rows = [7 + i % 8 for i in range(requests)]
    case = Case(rows, [60 + 17 * i for i in range(requests)], heads=4, kv_heads=1, dim=dim, group=dim, block=32, seed=6)
    total = sum(case.lens)
    fill(case, case.normal(total, dim), case.normal(total, dim))
    q = case.normal(case.T, 4 * dim)
    out, lse = case.attend(q)
    assert case.error() == 0
    check(case, q, out, lse)
