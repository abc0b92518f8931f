"""Products with 4-bit weights where sums that cancel would show: codes at and near their zero
point, one infinite or one very large x."""
import pytest

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
