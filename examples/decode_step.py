"""One decode step of one attention layer served to several adapters at once, every product of
it by the library's kernels: q, k and v by 4-bit weights (w4_matvec) with each request's LoRA
delta added (bgmv), rotary positions and the append to the 4-bit cache (kv_append), attention
over it (kv_attend), and the output projection with its delta.

The cache's blocks and the adapters' rows live in one pool of pages, as the unified pool is
meant: block b is a run of pool pages.

    python examples/decode_step.py            # a Llama-3-8B layer, 64 requests, in one CUDA graph, timed
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

import heterogeneous_adapters_gb300 as lora


class Layer:
    """Random weights, adapters and an empty cache of one layer, and a step over them."""

    def __init__(self, h=4096, heads=32, kv_heads=8, dim=128, requests=64, max_len=1024, adapters=16, rank=16,
                 weight_group=128, kv_group=128, block=64, seed=0):
        self.h, self.heads, self.kv_heads, self.dim, self.T = h, heads, kv_heads, dim, requests
        self.block, self.kv_group, self.weight_group, self.rank = block, kv_group, weight_group, rank
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        nq, nk = heads * dim, kv_heads * dim
        self.dims = [(h, nq), (h, nk), (h, nk), (nq, h)]            # q, k, v, o
        # 4-bit weights with a scale and a zero point per group
        self.weights = []
        for k, n in self.dims:
            codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8, device="cuda")
            scales = (torch.rand(k // weight_group, n, generator=g, device="cuda") * 0.2 + 0.1).div(k ** 0.5).half()
            zeros = torch.randint(0, 256, (k // weight_group, n // 2), generator=g, dtype=torch.uint8, device="cuda")
            self.weights.append((codes, scales, zeros))
        # the pool: adapter pages first, then the cache's blocks
        pages_of = lambda d: -(-d // h)  # noqa: E731
        per_layer = sum(pages_of(i) + pages_of(o) for i, o in self.dims)
        adapter_pages = adapters * per_layer * rank
        self.block_pages = -(-lora.kv_block_bytes(block, kv_heads, dim, kv_group) // (2 * h))
        self.max_blocks = -(-max_len // block)
        blocks = requests * self.max_blocks
        self.first_block = -(-adapter_pages // self.block_pages)
        self.pages = torch.empty((self.first_block + blocks) * self.block_pages, h, dtype=torch.bfloat16, device="cuda")
        self.pages[:adapter_pages] = (normal(adapter_pages, h) * 0.02).bfloat16()
        order = torch.randperm(adapter_pages, generator=g, device="cuda").int()
        self.page_table = order.contiguous()
        self.pt_off = (torch.arange(adapters, device="cuda") * per_layer * rank).long()
        self.ranks = torch.full((adapters,), rank, dtype=torch.int32, device="cuda")
        self.scales = torch.full((adapters,), 2.0, device="cuda")
        self.pool = lora.Pool(self.pages, self.pages.shape[0], h, self.page_table, self.page_table.numel(), self.pt_off, self.ranks,
                              self.scales, adapters, 1, 4, rank, proj_dims=self.dims)
        self.kv = lora.KvCache(self.pages, self.first_block + blocks, self.block_pages * 2 * h, block, kv_heads, dim, kv_group)
        self.table = (self.first_block + torch.randperm(blocks, generator=g, device="cuda")).int().view(requests, self.max_blocks)
        self.adapter = torch.randint(-1, adapters, (requests,), generator=g, device="cuda").int()
        self.kv_len = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.q_start = torch.arange(requests + 1, dtype=torch.int32, device="cuda")
        angle = np.arange(max_len)[:, None] * 500000.0 ** (-np.arange(0, dim, 2) / dim)[None]
        self.rope = lora.Rope(torch.tensor(np.cos(angle), dtype=torch.float32, device="cuda"),
                              torch.tensor(np.sin(angle), dtype=torch.float32, device="cuda"), max_len, dim, lora.LORA_ROPE_HALVES)
        # buffers and descriptions a server keeps
        self.x = torch.empty(requests, h, dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.empty(requests, nq + 2 * nk, dtype=torch.bfloat16, device="cuda")
        self.q = torch.empty(requests, nq, dtype=torch.bfloat16, device="cuda")
        self.att = torch.empty(requests, nq, dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty(requests, h, dtype=torch.bfloat16, device="cuda")
        self.parts = [self.qkv[:, :nq], self.qkv[:, nq:nq + nk], self.qkv[:, nq + nk:]]
        ld = self.qkv.shape[1]
        w4 = lambda x, y, ldy, i: (x, y, x.stride(0), ldy, *self.weights[i], self.dims[i][1], self.dims[i][0], weight_group)  # noqa: E731
        self.w_qkv = lora.w4_problems([w4(self.x, y, ld, i) for i, y in enumerate(self.parts)])
        self.w_out = lora.w4_problems([w4(self.att, self.out, h, 3)])
        self.d_qkv = [(self.x, y, h, ld, 0, i) for i, y in enumerate(self.parts)]
        self.d_out = [(self.att, self.out, nq, h, 0, 3)]
        self.batch = lora.KvBatch(self.q_start, self.kv_len, self.table, requests, requests, self.max_blocks, 1)
        self.ws_bytes = lora.workspace_size(self.pool, requests, requests)       # the delta's grouping
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")
        self.step_bytes = max(lora.kv_workspace_size(self.kv, self.batch, heads), lora.w4_workspace_size(self.w_qkv, requests))
        self.step_ws = torch.empty(self.step_bytes, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        lora.workspace_init(self.ws, self.ws_bytes, stream)
        lora.kv_workspace_init(self.step_ws, self.step_bytes, stream)
        torch.cuda.current_stream().synchronize()

        self.graph = None

    def step(self, x):
        """x bf16 [requests][h] -> the layer's attention output, the cache one token longer."""
        self.x.copy_(x)
        if self.graph is not None:
            self.graph.replay()
        else:
            self.calls()
        return self.out

    def capture(self):
        """Later steps replay one CUDA graph of the calls: their buffers stay where they are, and the
        lengths advance on the device."""
        side, lens = torch.cuda.Stream(), self.kv_len.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.calls()                        # loads the kernels; the next step writes the same token again
            self.kv_len.copy_(lens)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                self.calls()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = graph

    def calls(self):
        stream = torch.cuda.current_stream().cuda_stream
        ws, step = (self.ws, self.ws_bytes, stream), (self.step_ws, self.step_bytes, stream)
        self.kv_len += 1
        lora.w4_matvec(self.w_qkv, self.T, *step)
        lora.bgmv(self.pool, self.d_qkv, self.adapter, self.T, *ws)
        ld, nq = self.qkv.shape[1], self.heads * self.dim
        lora.kv_append(self.kv, self.batch, self.parts[0], ld, self.q, nq, self.heads, self.parts[1], ld, self.parts[2], ld, self.rope, *step)
        lora.kv_attend(self.kv, self.batch, self.q, nq, self.heads, self.dim ** -0.5, self.att, nq, None, *step)
        lora.w4_matvec(self.w_out, self.T, *step)
        lora.bgmv(self.pool, self.d_out, self.adapter, self.T, *ws)

    def errors(self):
        stream = torch.cuda.current_stream().cuda_stream
        return lora.get_device_error(self.ws, stream) | lora.get_device_error(self.step_ws, stream)


def main():
    layer = Layer()
    x = torch.randn(layer.T, layer.h, device="cuda").bfloat16()
    layer.capture()
    for _ in range(200):
        layer.step(x)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(100):
        layer.step(x)
    b.record()
    torch.cuda.synchronize()
    print(f"{layer.T} requests at {int(layer.kv_len[0])} tokens: {a.elapsed_time(b) * 10:.1f} us a step, device errors {layer.errors():#x}")


if __name__ == "__main__":
    main()
