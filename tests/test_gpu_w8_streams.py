"""Two 8-bit MLP layers (examples/mlp_step.py) at once on two streams, each with its buffers and workspaces: the
wide products of one beside the deltas, norms and activations of the other."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,segments", [(900, True), (200, True), (64, False), (9, False)])
def test_layers_on_two_streams(cuda, T, segments):
    from mlp_step import Mlp
    g = cuda.Generator(device="cuda").manual_seed(T)
    layers = [Mlp(1024, 2816, rows=T, adapters=4, rank=16, seed=i) for i in range(2)]
    ids = cuda.randint(-1, 4, (T,), generator=g, device="cuda").int()
    start = cuda.tensor([0, T // 3, T // 3 + 1, T], device="cuda").int()
    args = (None, start, cuda.tensor([2, -1, 3], device="cuda").int()) if segments else (ids,)
    inputs = [[cuda.randn(T, 1024, generator=g, device="cuda").bfloat16() for _ in range(2)] for _ in layers]
    want = []
    for layer, (x, res) in zip(layers, inputs):
        want.append([t.clone() for t in (layer.step(x, res, *args), layer.residual, layer.xa)])
        cuda.cuda.synchronize()
    streams = [cuda.cuda.Stream() for _ in layers]
    for _ in range(10):
        for layer in layers:
            layer.out.fill_(3)
        cuda.cuda.synchronize()
        for _ in range(3):
            for layer, stream, (x, res) in zip(layers, streams, inputs):
                with cuda.cuda.stream(stream):
                    layer.step(x, res, *args)
        cuda.cuda.synchronize()
        for layer, w in zip(layers, want):
            assert all(cuda.equal(a, b) for a, b in zip((layer.out[:T], layer.residual, layer.xa), w))
            assert layer.errors() == 0
