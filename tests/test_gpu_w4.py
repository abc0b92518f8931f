"""Products with 4-bit weights (include/lora_w4.h) against y = x W^T in 64 bits."""
import numpy as np
import pytest

import heterogeneous_adapters_gb300 as lora

pytestmark = pytest.mark.gpu


def problem(torch, g, T, N, K, group, zeros, pad=0, x=None):
    dev = dict(device="cuda")
    p = {"N": N, "K": K, "group": group, "T": T}
    p["x"] = x if x is not None else torch.randn(T, K + pad, generator=g, **dev).bfloat16()
    p["y"] = torch.full((T, N + pad), 7.0, dtype=torch.bfloat16, **dev)
    p["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, **dev)
    p["scales"] = (0.01 * (0.5 + torch.rand(K // group, N, generator=g, **dev))).half()
    p["scales"][0, :2] = -p["scales"][0, :2]
    p["zeros"] = torch.randint(0, 256, (K // group, N // 2), generator=g, dtype=torch.uint8, **dev) if zeros else None
    return p


def call(torch, ps, T):
    pr = lora.w4_problems([(p["x"], p["y"], p["x"].stride(0), p["y"].stride(0), p["codes"], p["scales"], p["zeros"], p["N"],
                            p["K"], p["group"]) for p in ps])
    size = lora.w4_workspace_size(pr, T)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    lora.kv_workspace_init(ws, size, stream)
    lora.w4_matvec(pr, T, ws, size, stream)
    first = [p["y"].clone() for p in ps]
    lora.w4_matvec(pr, T, ws, size, stream)                  # the same workspace again: the same bits
    for p, y in zip(ps, first):
        assert torch.equal(p["y"].view(torch.int16), y.view(torch.int16))
    assert lora.get_device_error(ws, stream) == 0


def check(torch, p):
    """bf16 rounds once (2^-8); an fp32 sum of exact products is within a few
    hundred roundings of sum |x w|: 2^-14."""
    T, N, K, G = p["T"], p["N"], p["K"], p["group"]
    c = torch.stack([p["codes"] & 15, p["codes"] >> 4], -1).view(N, K // G, G).double()
    z = 8.0
    if p["zeros"] is not None:
        z = torch.stack([p["zeros"] & 15, p["zeros"] >> 4], -1).view(K // G, N).t()[..., None].double()
    w = ((c - z) * p["scales"].t()[..., None].double()).view(N, K)
    x = p["x"][:, :K].double()
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    got = p["y"][:, :N].double()
    assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * size).all()), ((got - want).abs() / size).max()
    assert bool((p["y"][:, N:] == 7.0).all())


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 200, 256])
@pytest.mark.parametrize("N,K,group,zeros", [(256, 512, 128, True), (8, 32, 32, False), (200, 384, 64, True), (1032, 1152, 128, False),
                                             (136, 4160, 32, True), (1024, 4096, 128, True)])
def test_one_projection(cuda, T, N, K, group, zeros):
    g = cuda.Generator(device="cuda").manual_seed(T + N)
    p = problem(cuda, g, T, N, K, group, zeros, pad=8 * (T % 3))
    call(cuda, [p], T)
    check(cuda, p)


@pytest.mark.parametrize("T", [1, 5, 24, 64, 130])
def test_projections_of_different_shapes_in_one_call(cuda, T):
    g = cuda.Generator(device="cuda").manual_seed(T)
    a = problem(cuda, g, T, 512, 1024, 128, True)
    ps = [a, problem(cuda, g, T, 128, 1024, 128, False, x=a["x"]), problem(cuda, g, T, 264, 2048, 64, True, pad=16),
          problem(cuda, g, T, 40, 96, 32, True), problem(cuda, g, T, 2048, 256, 128, False)]
    call(cuda, ps, T)
    for p in ps:
        check(cuda, p)


@pytest.mark.parametrize("T", [1, 20, 64])
def test_model_widths(cuda, T):
    g = cuda.Generator(device="cuda").manual_seed(T)
    for N, K in ((4096, 14336), (14336, 4096), (5120, 5120)):
        p = problem(cuda, g, T, N, K, 128, True)
        call(cuda, [p], T)
        check(cuda, p)


@pytest.mark.parametrize("T", [1, 12, 64, 200])
def test_rows_do_not_mix(cuda, T):
    """A row of infinities or NaN leaves the other rows as they are."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, T, 256, 512, 128, True)
    call(cuda, [p], T)
    clean = p["y"].clone()
    bad = T // 2
    p["x"][bad] = float("inf")
    p["x"][bad, ::2] = float("nan")
    pr = lora.w4_problems([(p["x"], p["y"], 512, 256, p["codes"], p["scales"], p["zeros"], 256, 512, 128)])
    size = lora.w4_workspace_size(pr, T)
    ws = cuda.zeros(size, dtype=cuda.uint8, device="cuda")
    lora.w4_matvec(pr, T, ws, size, cuda.cuda.current_stream().cuda_stream)
    keep = [t for t in range(T) if t != bad]
    assert cuda.equal(p["y"][keep], clean[keep]) and bool(p["y"][bad].isnan().all())


def test_refusals(cuda):
    from heterogeneous_adapters_gb300 import _binding as B
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, 4, 64, 256, 64, True)
    ws = cuda.zeros(1 << 20, dtype=cuda.uint8, device="cuda")
    stream = cuda.cuda.current_stream().cuda_stream

    def status(T=4, size=1 << 20, n=1, **kw):
        a = dict(x=p["x"], y=p["y"], ldx=256, ldy=64, codes=p["codes"], scales=p["scales"], zeros=p["zeros"], N=64, K=256, group=64)
        a.update(kw)
        with pytest.raises(lora.LoraError) as e:
            lora.w4_matvec(lora.w4_problems([tuple(a.values())] * n), T, ws, size, stream)
        return e.value.status

    assert status(T=lora.LORA_W4_MAX_ROWS + 1) == B.LORA_ETOOBIG
    assert status(n=lora.LORA_W4_MAX_PROBLEMS + 1) == B.LORA_ETOOBIG
    assert status(size=0) == B.LORA_EWORKSPACE
    assert status(T=-1) == B.LORA_EINVAL
    assert status(N=60) == B.LORA_EINVAL
    assert status(group=48) == B.LORA_EINVAL
    assert status(K=200) == B.LORA_EINVAL
    assert status(ldx=248) == B.LORA_EINVAL
    assert status(ldy=63) == B.LORA_EALIGN
    assert status(x=None) == B.LORA_EINVAL
    assert status(codes=p["codes"].data_ptr() + 8) == B.LORA_EALIGN
    lora.w4_matvec(lora.w4_problems([]), 4, ws, 1 << 20, stream)
    assert bool((p["y"] == 7).all())
