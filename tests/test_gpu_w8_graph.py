"""An 8-bit MLP layer (examples/mlp_step.py) with a captured graph, called with other adapters than those it
was captured with."""
import os
import sys

import pytest

from .test_gpu_w8_step import check_layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 20, 64])
def test_replays_take_the_adapters_of_their_step(cuda, T):
    from mlp_step import Mlp
    mlp = Mlp(512, 1408, rows=T + 2, adapters=4, rank=8)
    g = cuda.Generator(device="cuda").manual_seed(T)
    first = cuda.randint(-1, 4, (T,), generator=g, device="cuda").int()
    mlp.capture(T, first)

    def step(adapters, *args):
        x, res = (cuda.randn(T, 512, generator=g, device="cuda").bfloat16() for _ in range(2))
        mlp.step(x, res, *args)
        assert mlp.errors() == 0
        check_layer(cuda, mlp, x, res, adapters)

    for adapter in (first, (first + 2) % 5 - 1, cuda.full_like(first, -1), first.flip(0)):
        step(adapter.tolist(), adapter)
        held = adapter.clone()
        held[0] = (int(held[0]) + 2) % 5 - 1                       # the caller's tensor written anew
        adapter.copy_(held)
        step(held.tolist(), adapter)
    # prompts of as many rows
    start, which = cuda.tensor([0, T], device="cuda").int(), cuda.tensor([3], device="cuda").int()
    step([3] * T, None, start, which)
    step(first.tolist(), first)
