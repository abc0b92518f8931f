"""Rows left in 8 bits (include/lora_w8.h) in arrays whose offsets pass 32 bits: wide pitches and many rows."""
import pytest

import heterogeneous_adapters_gb300 as lora

from .test_gpu_q8 import ACTS

pytestmark = pytest.mark.gpu


def stream(torch):
    return torch.cuda.current_stream().cuda_stream


def test_pitches_past_32_bits(cuda):
    """Nine rows half a billion values apart: the bits of rows that lie side by side."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    T, pitch = 9, 2 ** 29 + 16
    wide = [cuda.empty(T * pitch, dtype=cuda.bfloat16, device="cuda").view(T, pitch) for _ in range(3)]
    codes = cuda.empty(T * pitch, dtype=cuda.int8, device="cuda").view(T, pitch)
    for d in (64, 8192):
        x, r = (cuda.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
        w = cuda.randn(d, generator=g, device="cuda").bfloat16()
        want = [cuda.empty_like(x), cuda.empty_like(x), cuda.empty(T, d, dtype=cuda.int8, device="cuda"), cuda.empty(T, device="cuda")]
        scales = cuda.empty(T, device="cuda")

        def check():
            for a, b in ((wide[1][:, :d], want[0]), (wide[2][:, :d], want[1]), (codes[:, :d], want[2]), (scales, want[3])):
                assert cuda.equal(a, b)

        lora.q8_norm(lora.Q8Norm(x, d, r, d, want[0], d, w, 1e-5, d, lora.Q8Rows(want[2], d, want[3], want[1], d)), T, stream(cuda))
        wide[0][:, :d], wide[1][:, :d] = x, r                      # the sum in the residual's place
        rows = lora.Q8Rows(codes, pitch, scales, wide[2], pitch)
        lora.q8_norm(lora.Q8Norm(wide[0], pitch, wide[1], pitch, wide[1], pitch, w, 1e-5, d, rows), T, stream(cuda))
        check()
        for act in ACTS.values():
            lora.q8_gate(lora.Q8Gate(x, d, r, d, act, d, lora.Q8Rows(want[2], d, want[3], want[1], d)), T, stream(cuda))
            want[0].copy_(r)
            wide[0][:, :d], wide[1][:, :d] = x, r
            lora.q8_gate(lora.Q8Gate(wide[0], pitch, wide[1], pitch, act, d, rows), T, stream(cuda))
            check()


def test_the_most_rows(cuda):
    """2^24 rows: any of them are as in a call of their own."""
    g = cuda.Generator(device="cuda").manual_seed(2)
    T, d = lora.LORA_Q8_MAX_ROWS, 272                              # 4.6 billion values
    x = cuda.empty(T, d, dtype=cuda.bfloat16, device="cuda")
    for at in range(0, T, T // 16):
        x[at:at + T // 16].copy_(cuda.randn(T // 16, d, generator=g, device="cuda"))
    w = cuda.randn(d, generator=g, device="cuda").bfloat16()
    out = (cuda.empty(T, d, dtype=cuda.int8, device="cuda"), cuda.empty(T, device="cuda"), cuda.empty_like(x))

    def norm(x, out, n):
        lora.q8_norm(lora.Q8Norm(x, d, None, 0, None, 0, w, 1e-5, d, lora.Q8Rows(out[0], d, out[1], out[2], d)), n, stream(cuda))

    def gate(x, out, n):
        lora.q8_gate(lora.Q8Gate(x, d, x, d, lora.LORA_ACT_SILU, d, lora.Q8Rows(out[0], d, out[1], out[2], d)), n, stream(cuda))

    for f in (norm, gate):
        f(x, out, T)
        for first in (0, 2 ** 31 // d - 50, 2 ** 32 // d - 50, T - 100):
            few = tuple(cuda.empty_like(o[:100]) for o in out)
            f(x[first:first + 100], few, 100)
            assert all(cuda.equal(a, o[first:first + 100]) for a, o in zip(few, out))
