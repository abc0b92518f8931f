"""Attention over the 4-bit cache where a visible token is not a number; against 64 bits with the
bounds of tests/kv_exact.py."""
import numpy as np
import pytest

import heterogeneous_adapters_gb300 as lora

from .kv_exact import check
from .test_gpu_kv import Case

pytestmark = pytest.mark.gpu

FORMS = [(64, 64), (64, 32), (128, 128), (128, 32)]


def fill(case, k, v):
    """Every token of every request: k, v [tokens][kv heads * D], appended as they are."""
    t = case.torch
    start = t.tensor(np.concatenate([[0], np.cumsum(case.lens)]), dtype=t.int32, device="cuda")
    total = sum(case.lens)
    batch = lora.KvBatch(start, case.kv_len, case.table, case.n, total, case.max_blocks, max(case.lens))
    lora.kv_append(case.kv, batch, None, 0, None, 0, 0, k, k.shape[1], v, v.shape[1], case.rope(0), case.ws, case.size, case.stream)


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
