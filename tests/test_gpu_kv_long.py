"""Sizes at which the loops of the 4-bit cache's kernels run long: contexts of which a warp takes
more steps than it looks tiles up for at once, and batches of rows large enough that a warp
appends and reads back many heads, from queries through keys to values."""
import numpy as np
import pytest

from .kv_exact import check
from .test_gpu_kv import KV, Case, check_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (128, 32)])
@pytest.mark.parametrize("missing", [False, True])
def test_attend_contexts_of_many_steps_a_warp(cuda, dim, group, missing):
    case = Case([1, 1, 2], [200003, 199999, 131103], heads=8, kv_heads=8, dim=dim, group=group, block=64, seed=1)
    case.fill()
    if missing:
        case.table[0, 40:43] = -1
        case.table[1, 3000] = case.blocks + 7
    q = case.normal(case.T, 8 * dim)
    out, lse = case.attend(q)
    assert case.error() == (KV if missing else 0)
    if missing:
        case.table[1, 3000] = -1
    check(case, q, out, lse, heads=[0, 5])


@pytest.mark.parametrize("shape", [dict(heads=32, kv_heads=8, dim=128, group=128, block=64), dict(heads=5, kv_heads=5, dim=128, group=32, block=16),
                                   dict(heads=16, kv_heads=4, dim=64, group=64, block=32), dict(heads=7, kv_heads=7, dim=64, group=32, block=48)])
@pytest.mark.parametrize("style", [0, 1])
def test_append_and_read_of_many_rows(cuda, shape, style):
    rows, lens = [1500, 3000, 1, 499], [1500, 3100, 77, 2000]
    case = Case(rows, lens, seed=style, **shape)
    D, a, b = case.dim, case.heads * case.dim, (case.heads + case.kv_heads) * case.dim
    qkv = case.normal(case.T, (case.heads + 2 * case.kv_heads) * D)
    q, k, v = qkv[:, :a], qkv[:, a:b], qkv[:, b:]
    out = case.append(q, k, v, case.rope(style=style))
    assert case.error() == 0
    check_append(case, q, k, v, out, np.concatenate([np.arange(n - m, n) for m, n in zip(rows, lens)]), D, style)
