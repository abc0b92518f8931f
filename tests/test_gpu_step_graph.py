"""The decode step of examples/decode_step.py captured in a CUDA graph and replayed, against the
same calls made one by one."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [dict(h=512, heads=8, kv_heads=2, dim=128, kv_group=128, block=32, requests=5),
                                   dict(h=1024, heads=6, kv_heads=3, dim=64, kv_group=32, block=16, requests=40)])
def test_replayed_steps_are_the_calls(cuda, shape):
    from decode_step import Layer
    eager, graph = (Layer(max_len=64, adapters=3, rank=8, weight_group=64, **shape) for _ in range(2))
    g = cuda.Generator(device="cuda").manual_seed(7)
    for step in range(24):
        if step == 3:
            graph.capture()
        x = cuda.randn(eager.T, eager.h, generator=g, device="cuda").bfloat16()
        a, b = eager.step(x), graph.step(x)
        assert cuda.equal(a.view(cuda.int16), b.view(cuda.int16)), step
        assert cuda.equal(eager.kv_len, graph.kv_len) and int(graph.kv_len[0]) == step + 1
    assert eager.errors() == 0 and graph.errors() == 0
    # the caches hold the same tokens (bytes of places that hold none are the pools' own)
    assert cuda.equal(eager.table, graph.table)
    held = eager.table[:, 0].long()
    blocks = [layer.pages.view(-1, layer.block_pages * layer.h)[held].view(cuda.uint8) for layer in (eager, graph)]
    tile = 16 * eager.dim                                             # codes of the first 16 tokens of KV head 0
    assert cuda.equal(blocks[0][:, :tile], blocks[1][:, :tile])
