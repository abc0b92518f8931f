"""The MLP of one layer of an 8-bit base model served to several adapters at once: the residual's
addition and the norm (q8_norm), the two wide projections in 8 bits (w8_matmul) with each
request's LoRA delta added, the gated activation (q8_gate), and the last projection with its
delta.  The rows may be a decode step's, one for each request (bgmv), or prompts (sgmv).

    python examples/mlp_step.py            # a Llama-3-8B layer: 64 requests in one CUDA graph, and 2,000 rows of prompts, timed
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import heterogeneous_adapters_gb300 as lora


class Mlp:
    """Random weights and adapters of one layer, and a step over up to `rows` rows."""

    def __init__(self, h=4096, f=14336, rows=64, adapters=16, rank=16, seed=0):
        self.h, self.f, self.rows, self.rank = h, f, rows, rank
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.dims = [(h, f), (h, f), (f, h)]                        # gate, up, down
        # 8-bit weights with a scale per channel
        self.weights = []
        for k, n in self.dims:
            w = normal(n, k)
            top = w.abs().amax(1)
            self.weights.append((torch.round(w * (127 / top)[:, None]).to(torch.int8), top / 127 / k ** 0.5))
        self.norm = (1 + 0.1 * normal(h)).bfloat16()
        pages_of = lambda d: -(-d // h)  # noqa: E731
        per_layer = sum(pages_of(i) + pages_of(o) for i, o in self.dims)
        self.pages = (normal(adapters * per_layer * rank, h) * 0.02).bfloat16()
        self.page_table = torch.randperm(self.pages.shape[0], generator=g, device="cuda").int()
        self.pt_off = (torch.arange(adapters, device="cuda") * per_layer * rank).long()
        self.ranks = torch.full((adapters,), rank, dtype=torch.int32, device="cuda")
        self.scales = torch.full((adapters,), 2.0, device="cuda")
        self.pool = lora.Pool(self.pages, self.pages.shape[0], h, self.page_table, self.page_table.numel(), self.pt_off, self.ranks,
                              self.scales, adapters, 1, 3, rank, proj_dims=self.dims)
        # buffers and descriptions a server keeps
        bf = lambda d: torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.adapter = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        self.x, self.residual, self.xn, self.xa, self.out = bf(h), bf(h), bf(h), bf(f), bf(h)
        self.both = bf(2 * f)                                       # gate and up, side by side
        self.q, self.qs = torch.empty(rows, h, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        self.qa, self.qas = torch.empty(rows, f, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        gate, up = self.both[:, :f], self.both[:, f:]
        # the residual stream is held in place
        self.call_norm = lora.Q8Norm(self.x, h, self.residual, h, self.residual, h, self.norm, 1e-5, h, lora.Q8Rows(self.q, h, self.qs, self.xn, h))
        self.call_gate = lora.Q8Gate(gate, 2 * f, up, 2 * f, lora.LORA_ACT_SILU, f, lora.Q8Rows(self.qa, f, self.qas, self.xa, f))
        self.w_wide = lora.w8_problems([(self.q, self.qs, y, h, 2 * f, *self.weights[i], f, h) for i, y in enumerate((gate, up))])
        self.w_down = lora.w8_problems([(self.qa, self.qas, self.out, f, h, *self.weights[2], h, f)])
        self.d_wide = [(self.xn, y, h, 2 * f, 0, i) for i, y in enumerate((gate, up))]
        self.d_down = [(self.xa, self.out, f, h, 0, 2)]
        self.ws_bytes = lora.workspace_size(self.pool, rows, rows)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")
        self.step_bytes = max(lora.w8_workspace_size(self.w_wide, rows), lora.w8_workspace_size(self.w_down, rows))
        self.step_ws = torch.empty(self.step_bytes, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        lora.workspace_init(self.ws, self.ws_bytes, stream)
        lora.kv_workspace_init(self.step_ws, self.step_bytes, stream)
        torch.cuda.current_stream().synchronize()
        self.graph = None

    def calls(self, T, adapter=None, seg_start=None, seg_adapter=None):
        """Rows 0 .. T - 1: each with the adapter of `adapter`, or in segments."""
        stream = torch.cuda.current_stream().cuda_stream
        ws, step = (self.ws, self.ws_bytes, stream), (self.step_ws, self.step_bytes, stream)

        def delta(problems):
            if seg_start is None:
                lora.bgmv(self.pool, problems, adapter, T, *ws)
            else:
                lora.sgmv(self.pool, problems, seg_start, seg_adapter, seg_adapter.numel(), T, *ws)

        lora.q8_norm(self.call_norm, T, stream)
        lora.w8_matmul(self.w_wide, T, *step)
        delta(self.d_wide)
        lora.q8_gate(self.call_gate, T, stream)
        lora.w8_matmul(self.w_down, T, *step)
        delta(self.d_down)

    def step(self, x, residual, *adapters):
        """x, residual bf16 [T][h] -> what the MLP adds to the residual stream, which self.residual holds."""
        T = x.shape[0]
        self.x[:T].copy_(x)
        self.residual[:T].copy_(residual)
        if self.graph is not None and T == self.graph[1] and len(adapters) == 1:
            self.adapter[:T].copy_(adapters[0])
            self.graph[0].replay()
        else:
            self.calls(T, *adapters)
        return self.out[:T]

    def capture(self, T, adapter):
        """Later steps of T requests replay one CUDA graph of the calls, each with the adapters it is given."""
        self.adapter[:T].copy_(adapter)
        side, held = torch.cuda.Stream(), self.residual.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.calls(T, self.adapter[:T])                         # loads the kernels
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                self.calls(T, self.adapter[:T])
            self.residual.copy_(held)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = graph, T

    def errors(self):
        stream = torch.cuda.current_stream().cuda_stream
        return lora.get_device_error(self.ws, stream) | lora.get_device_error(self.step_ws, stream)


def main():
    rows = 2000
    mlp = Mlp(rows=rows)
    x, residual = (torch.randn(rows, mlp.h, device="cuda").bfloat16() for _ in range(2))
    adapter = torch.randint(-1, 16, (64,), device="cuda").int()
    mlp.capture(64, adapter)
    start = torch.tensor([0, 700, 701, 1500, rows], dtype=torch.int32, device="cuda")
    which = torch.tensor([3, -1, 0, 7], dtype=torch.int32, device="cuda")
    for name, T, args in (("64 requests, one graph", 64, (adapter,)), ("2,000 rows of prompts", rows, (None, start, which))):
        for _ in range(20):
            mlp.step(x[:T], residual[:T], *args)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(100):
            mlp.step(x[:T], residual[:T], *args)
        b.record()
        torch.cuda.synchronize()
        print(f"{name}: {a.elapsed_time(b) * 10:.1f} us a step, device errors {mlp.errors():#x}")


if __name__ == "__main__":
    main()
