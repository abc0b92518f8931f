"""Products of 8-bit integers (include/lora_w8.h) to the bit: the whole sum in fp32, times the row's
scale, times the channel's, rounded to bf16 once; and arrays whose offsets pass 32 bits."""
import pytest

import heterogeneous_adapters_gb300 as lora

from .test_gpu_w8 import call, codes, problem, problems, workspace

pytestmark = pytest.mark.gpu


def want(torch, p):
    T, N, K = p["T"], p["N"], p["K"]
    x, out = p["x"][:T, :K].double(), []
    for at in range(0, N, 8192):
        out.append(x @ p["w"][at:at + 8192].double().t())          # whole numbers under 2^53
    s = torch.cat(out, 1)
    return s, (s.float() * p["xs"][:, None] * p["ws"]).bfloat16()


def check_bits(torch, p, most=2 ** 24):
    s, y = want(torch, p)
    assert most is None or float(s.abs().max()) <= most
    assert torch.equal(p["y"][:p["T"], :p["N"]].contiguous().view(torch.int16), y.view(torch.int16))
    assert bool((p["y"][p["T"]:] == 7.0).all()) and bool((p["y"][:, p["N"]:] == 7.0).all())


@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 33, 64, 65, 129, 257, 700])
@pytest.mark.parametrize("N,K", [(8, 16), (264, 528), (4096, 1024), (5128, 5136), (392, 65536), (8200, 4112)])
def test_bits(cuda, T, N, K):
    g = cuda.Generator(device="cuda").manual_seed(T + N)
    p = problem(cuda, g, T, N, K, pad=8 * (T % 3))
    call(cuda, [p], T)
    check_bits(cuda, p)


@pytest.mark.parametrize("T", [1, 8, 9, 40, 64, 300])
@pytest.mark.parametrize("N", [40, 16392])
@pytest.mark.parametrize("a,b", [(127, 127), (-127, 127), (-128, 127), (-128, -128)])
def test_bits_of_sums_up_to_2_to_the_24(cuda, T, N, a, b):
    """Every product the largest: 1,024 of them are at most 2^24, and both kernels hold each sum on the way."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, T, N, 1024)
    p["x"].fill_(a)
    p["w"].fill_(b)
    call(cuda, [p], T)
    check_bits(cuda, p)


@pytest.mark.parametrize("T", [1, 5, 8])
@pytest.mark.parametrize("K", [1040, 16384, lora.LORA_W8_MAX_K])
@pytest.mark.parametrize("a,b", [(-128, -128), (-128, 127), (127, 127)])
def test_few_rows_sum_as_integers(cuda, T, K, a, b):
    """Up to 8 rows, always the few-row kernel, sums past 2^24 are whole numbers too, rounded once to fp32."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, T, 40, K)
    p["x"].fill_(a)
    p["w"].fill_(b)
    p["w"].view(-1)[::7] -= 1 if b > 0 else -1                     # sums that fp32 does not hold
    call(cuda, [p], T)
    check_bits(cuda, p, None)


@pytest.mark.parametrize("T", [3, 14, 40, 300])
def test_the_most_projections(cuda, T):
    """Sixteen projections, each with an x of its own, of unlike sizes."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    ps = [problem(cuda, g, T, 8 * (5 + 37 * i % 101), 16 * (1 + 29 * i % 67), pad=8 * (i % 2)) for i in range(lora.LORA_W8_MAX_PROBLEMS)]
    for more in ([], [problem(cuda, g, T, 12296, 5136)]):          # the second time one that takes the call to the other kernel
        ps[:len(more)] = more
        call(cuda, ps, T)
        for p in ps:
            check_bits(cuda, p)


@pytest.mark.parametrize("T", [8, 14, 40, 300])
def test_pitches_past_32_bits(cuda, T):
    """Rows of x and y whose offsets pass 2^32."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    pitch = (2 ** 32 // (T - 1) + 16) // 16 * 16
    for N, K in ((264, 1040), (8200, 4112)):
        p = problem(cuda, g, T, N, K)
        x, y = cuda.empty(T * pitch, dtype=cuda.int8, device="cuda").view(T, pitch), cuda.empty(T * pitch, dtype=cuda.bfloat16, device="cuda").view(T, pitch)
        x[:, :K + 16] = 99
        x[:, :K] = p["x"]
        y[:, :N + 8] = 7
        pr = lora.w8_problems([(x, p["xs"], y, pitch, pitch, p["w"], p["ws"], N, K)])
        ws, size = workspace(cuda, pr, T)
        lora.w8_matmul(pr, T, ws, size, cuda.cuda.current_stream().cuda_stream)
        p["y"] = y[:, :N + 8]
        check_bits(cuda, p)
        del x, y


@pytest.mark.parametrize("T", [1, 8, 40])
def test_weights_past_32_bits(cuda, T):
    """W of 4.5 GB."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    p = problem(cuda, g, T, 69128, 65536)
    call(cuda, [p], T)
    check_bits(cuda, p)
