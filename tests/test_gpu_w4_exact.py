"""Products with 4-bit weights where sums that cancel would show: codes at and near their zero
point, one infinite or one very large x."""
import pytest

import heterogeneous_adapters_gb300 as lora

from .test_gpu_w4 import call, problem

pytestmark = pytest.mark.gpu

ROWS = [1, 5, 8, 9, 16, 17, 64]


def weights(torch, p):
    """W in 64 bits."""
    N, K, G = p["N"], p["K"], p["group"]
    c = torch.stack([p["codes"] & 15, p["codes"] >> 4], -1).view(N, K // G, G).double()
    z = 8.0
    if p["zeros"] is not None:
        z = torch.stack([p["zeros"] & 15, p["zeros"] >> 4], -1).view(K // G, N).t()[..., None].double()
    return ((c - z) * p["scales"].t()[..., None].double()).view(N, K)


def at_zero(torch, p):
    """Every code set to its zero point."""
    N, K, G = p["N"], p["K"], p["group"]
    z = torch.full((N, K), 8, dtype=torch.uint8, device="cuda")
    if p["zeros"] is not None:
        z = torch.stack([p["zeros"] & 15, p["zeros"] >> 4], -1).view(K // G, N).t().repeat_interleave(G, 1)
    p["codes"].copy_(z[:, 0::2] | z[:, 1::2] << 4)


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_codes_at_their_zero_point(cuda, T, group, zeros):
    """Weights of zero give zeros, and four weights a row give their four products."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    p = problem(cuda, g, T, 264, 1024, group, zeros)
    # a mean that is not zero, and sizes that an fp32 sum has to round
    p["x"] = ((p["x"].float() + 3) * 2.0 ** (12 * cuda.rand(T, 1024, generator=g, device="cuda"))).bfloat16()
    at_zero(cuda, p)
    call(cuda, [p], T)
    assert not bool(p["y"].any())
    for j in range(4):
        p["codes"][:, 100 * j] ^= 1 + (j & 1) * 16
    call(cuda, [p], T)
    w, x = weights(cuda, p), p["x"].double()
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    # bf16 (2^-8), and fp32 sums of a few terms that are not zero
    assert bool(((p["y"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all())


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("zeros", [True, False])
def test_one_infinite_x(cuda, T, zeros):
    """An infinity times a weight is an infinity of its sign, and not a number where the weight is zero."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    p = problem(cuda, g, T, 136, 512, 64, zeros)
    p["scales"].abs_()
    bad = T // 2
    p["x"][bad, 77] = float("inf")
    call(cuda, [p], T)
    w = weights(cuda, p)[:, 77]
    y = p["y"].float()
    assert bool((y[bad][w > 0] == float("inf")).all()) and bool((y[bad][w < 0] == -float("inf")).all())
    assert bool(y[bad][w == 0].isnan().all())
    keep = [t for t in range(T) if t != bad]
    assert bool(y[keep].isfinite().all())


@pytest.mark.parametrize("T", ROWS)
def test_large_x(cuda, T):
    """Sums of code differences times x stay finite while they fit fp32."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    p = problem(cuda, g, T, 136, 512, 128, True)
    p["x"] = (p["x"].float().abs() * 2.0 ** 116).bfloat16()        # a group's sum of |code - zero| x is about 2^126
    call(cuda, [p], T)
    w, x = weights(cuda, p), p["x"].double()
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    assert bool(((p["y"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * size).all())


@pytest.mark.parametrize("T,block", [(17, 20), (64, 20), (64, 33), (128, 1000)])
def test_the_workspace_serves_on_after_a_wait_that_ran_out(cuda, T, block):
    """Row tiles shared by neighbouring workers, one of which never gets its codes: the timeout bit,
    and later calls on the same workspace are as on a fresh one."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    p = problem(cuda, g, T, 14336, 4096, 128, True)
    tup = lambda y: (p["x"], y, 4096, 14336, p["codes"], p["scales"], p["zeros"], 14336, 4096, 128)  # noqa: E731
    y = cuda.empty(T, 14336, dtype=cuda.bfloat16, device="cuda")
    pr, want = lora.w4_problems([tup(y)]), lora.w4_problems([tup(p["y"])])
    size, stream = lora.w4_workspace_size(pr, T), cuda.cuda.current_stream().cuda_stream
    ws, fresh = (cuda.zeros(size, dtype=cuda.uint8, device="cuda") for _ in range(2))
    lora.debug_w4_lost_block(pr, T, block, 5_000_000, ws, size, stream)
    assert lora.get_device_error(ws, stream) == 0x20
    for _ in range(3):
        p["x"].copy_(cuda.randn(T, 4096, generator=g, device="cuda").bfloat16())
        lora.w4_matvec(pr, T, ws, size, stream)
        lora.w4_matvec(want, T, fresh, size, stream)
        assert lora.get_device_error(ws, stream) == 0
        assert cuda.equal(y.view(cuda.int16), p["y"].view(cuda.int16))


def test_lost_block_refusals(cuda):
    from heterogeneous_adapters_gb300 import _binding as B
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, 20, 64, 256, 64, True)
    pr = lora.w4_problems([(p["x"], p["y"], 256, 64, p["codes"], p["scales"], p["zeros"], 64, 256, 64)])
    ws = cuda.zeros(lora.w4_workspace_size(pr, 20), dtype=cuda.uint8, device="cuda")
    for T, block, limit, want in ((16, 0, 5_000_000, B.LORA_EINVAL), (20, -1, 5_000_000, B.LORA_EINVAL),
                                  (20, 0, 1000, B.LORA_EINVAL), (20, 0, 3_000_000_000, B.LORA_ETOOBIG)):
        with pytest.raises(lora.LoraError) as e:
            lora.debug_w4_lost_block(pr, T, block, limit, ws, ws.numel(), 0)
        assert e.value.status == want
    assert bool((p["y"] == 7).all())
