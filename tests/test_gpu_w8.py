"""Products of 8-bit integers with scales per row and channel (include/lora_w8.h) against their
definition in 64 bits."""
import pytest

import heterogeneous_adapters_gb300 as lora

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 191, 200, 256, 257, 300, 512, 513, 1000]
SHAPES = [(8, 16), (24, 80), (136, 64), (200, 1040), (264, 528), (1032, 1152), (512, 4096)]


def codes(torch, g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def problem(torch, g, T, N, K, pad=0, x=None):
    """Two rows behind the last one and `pad` columns of y stay as they are."""
    p = {"T": T, "N": N, "K": K}
    p["x"] = x["x"] if x else codes(torch, g, T, K + 16 * (pad > 0))
    p["xs"] = x["xs"] if x else 0.01 + torch.rand(T, generator=g, device="cuda")
    p["w"] = codes(torch, g, N, K)
    p["ws"] = (torch.rand(N, generator=g, device="cuda") - 0.3) * 0.01
    p["y"] = torch.full((T + 2, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    return p


def problems(ps):
    return lora.w8_problems([(p["x"], p["xs"], p["y"], p["x"].stride(0), p["y"].stride(0), p["w"], p["ws"], p["N"], p["K"]) for p in ps])


def workspace(torch, pr, T):
    size = lora.w8_workspace_size(pr, T)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    lora.kv_workspace_init(ws, size, torch.cuda.current_stream().cuda_stream)
    return ws, size


def call(torch, ps, T):
    pr = problems(ps)
    ws, size = workspace(torch, pr, T)
    stream = torch.cuda.current_stream().cuda_stream
    lora.w8_matmul(pr, T, ws, size, stream)
    first = [p["y"].clone() for p in ps]
    lora.w8_matmul(pr, T, ws, size, stream)                  # the same workspace again: the same bits
    for p, y in zip(ps, first):
        assert torch.equal(p["y"].view(torch.int16), y.view(torch.int16))
    assert lora.get_device_error(ws, stream) == 0


def check(torch, p):
    """Sums under 2^24 are whole numbers that fp32 holds; two products with scales and the rounding to bf16."""
    T, N, K = p["T"], p["N"], p["K"]
    s = p["x"][:T, :K].double() @ p["w"].double().t()
    assert float(s.abs().max()) < 2 ** 24
    want = s * p["xs"].double()[:, None] * p["ws"].double()
    got = p["y"][:T, :N].double()
    assert bool(((got - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs()).all())
    assert bool((p["y"][T:] == 7.0).all()) and bool((p["y"][:, N:] == 7.0).all())


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("N,K", SHAPES)
def test_one_projection(cuda, T, N, K):
    g = cuda.Generator(device="cuda").manual_seed(T + N)
    p = problem(cuda, g, T, N, K, pad=8 * (T % 3))
    call(cuda, [p], T)
    check(cuda, p)


@pytest.mark.parametrize("T", [33, 40, 64, 65, 100, 128, 129, 200, 256, 257, 300, 520])
@pytest.mark.parametrize("N,K", [(8200, 4112), (6152, 4880), (16392, 2064), (65544, 400), (392, 65536)])
def test_one_large_projection(cuda, T, N, K):
    """W of 25 MB and more, its last tiles and its last block of K not full."""
    g = cuda.Generator(device="cuda").manual_seed(T + N)
    p = problem(cuda, g, T, N, K, pad=8 * (T % 3))
    call(cuda, [p], T)
    check(cuda, p)



@pytest.mark.parametrize("T", [5000, 40001, lora.LORA_W8_MAX_ROWS])
@pytest.mark.parametrize("N,K", [(8, 16), (264, 80), (520, 1040)])
def test_the_most_rows(cuda, T, N, K):
    g = cuda.Generator(device="cuda").manual_seed(T + N)
    p = problem(cuda, g, T, N, K, pad=8)
    call(cuda, [p], T)
    check(cuda, p)


@pytest.mark.parametrize("T", [1, 5, 24, 40, 64, 130, 257, 700])
def test_projections_of_different_shapes_in_one_call(cuda, T):
    g = cuda.Generator(device="cuda").manual_seed(T)
    a = problem(cuda, g, T, 512, 1024)
    ps = [a, problem(cuda, g, T, 128, 1024, x=a), problem(cuda, g, T, 264, 2048, pad=16), problem(cuda, g, T, 40, 96),
          problem(cuda, g, T, 2048, 256), problem(cuda, g, T, 8, 16)]
    call(cuda, ps, T)
    for p in ps:
        check(cuda, p)
    # the same behind one that takes the call to the other kernel
    ps.insert(1, problem(cuda, g, T, 6152, 4880))
    call(cuda, ps, T)
    for p in ps:
        check(cuda, p)


@pytest.mark.parametrize("T", [1, 20, 64, 150, 333, 2050])
def test_model_widths(cuda, T):
    g = cuda.Generator(device="cuda").manual_seed(T)
    for N, K in ((4096, 14336), (14336, 4096), (5120, 5120), (1024, 4096)):
        p = problem(cuda, g, T, N, K)
        call(cuda, [p], T)
        check(cuda, p)


@pytest.mark.parametrize("T", [1, 8, 13, 16, 20, 32, 33, 70])
@pytest.mark.parametrize("N,K", [(264, 1040), (4096, 1024), (40, 96), (512, 4096)])
def test_rows_at_any_multiple_of_16_bytes(cuda, T, N, K):
    """Rows that begin 16 bytes past a multiple of 32, of x, of W or of both, give the bits of rows that do not."""
    g = cuda.Generator(device="cuda").manual_seed(T + K)
    a = problem(cuda, g, T, N, K)
    call(cuda, [a], T)
    check(cuda, a)
    for move_x, move_w, pad in ((True, False, 0), (False, True, 0), (False, False, 16), (True, True, 32)):
        b = dict(a, y=cuda.full_like(a["y"], 7.0))
        store = cuda.full((T * (K + pad) + 32,), 99, dtype=cuda.int8, device="cuda")
        b["x"] = store[16 * move_x:][:T * (K + pad)].view(T, K + pad)
        b["x"][:, :K] = a["x"][:, :K]
        store = cuda.full((N * K + 32,), 99, dtype=cuda.int8, device="cuda")
        b["w"] = store[16 * move_w:][:N * K].view(N, K)
        b["w"].copy_(a["w"])
        call(cuda, [b], T)
        assert cuda.equal(a["y"].view(cuda.int16), b["y"].view(cuda.int16))


@pytest.mark.parametrize("T", [1, 12, 40, 64, 200, 300])
@pytest.mark.parametrize("a,b", [(-128, -128), (-128, 127), (127, 127)])
def test_largest_codes(cuda, T, a, b):
    """Sums far past 2^24: up to 32 rows they stay whole numbers, beyond they are fp32 sums."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    for K in (1024, 16384, lora.LORA_W8_MAX_K):
        p = problem(cuda, g, T, 40, K)
        p["x"].fill_(a)
        p["w"].fill_(b)
        call(cuda, [p], T)
        want = float(a * b * K) * p["xs"].double()[:, None] * p["ws"].double()
        # an fp32 sum of K terms of one sign: each of the additions of 16 terms may lose 2^-23 of the sum so far,
        # on the average of them half of that
        tol = 2.0 ** -8 + 2.0 ** -21 + K / 16 * 2.0 ** -24
        assert bool(((p["y"][:T].double() - want).abs() <= tol * want.abs()).all())


@pytest.mark.parametrize("T", [1, 12, 40, 64, 200, 300])
def test_rows_do_not_mix(cuda, T):
    """A row whose scale is not a number leaves the other rows as they are, a channel's the other channels."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, T, 264, 512)
    call(cuda, [p], T)
    clean, bad = p["y"].clone(), T // 2
    p["xs"][bad] = float("nan")
    p["ws"][100] = float("inf")
    call(cuda, [p], T)
    keep, cols = [t for t in range(T) if t != bad], [n for n in range(264) if n != 100]
    assert cuda.equal(p["y"][keep][:, cols], clean[keep][:, cols]) and bool(p["y"][bad].isnan().all())
    assert not bool(p["y"][keep][:, 100].isfinite().any())


def test_rows_and_channels_of_zeros(cuda):
    g = cuda.Generator(device="cuda").manual_seed(1)
    for T in (3, 40, 300):
        p = problem(cuda, g, T, 72, 272)
        p["x"][1] = 0
        p["w"][5] = 0
        call(cuda, [p], T)
        assert not bool(p["y"][1].any()) and not bool(p["y"][:T, 5].any())
        check(cuda, p)


def test_a_workspace_serves_fewer_rows(cuda):
    """One workspace, calls of many and of few rows in turn."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    big = problem(cuda, g, 700, 264, 1040)
    ws, size = workspace(cuda, problems([big]), 700)
    for T in (700, 3, 300, 40, 1, 700):
        p = problem(cuda, g, T, 264, 1040)
        lora.w8_matmul(problems([p]), T, ws, size, cuda.cuda.current_stream().cuda_stream)
        check(cuda, p)


def test_no_rows(cuda):
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, 4, 64, 256)
    ws, size = workspace(cuda, problems([p]), 4)
    lora.w8_matmul(problems([p]), 0, ws, size, cuda.cuda.current_stream().cuda_stream)
    lora.w8_matmul(lora.w8_problems([]), 4, ws, size, cuda.cuda.current_stream().cuda_stream)
    assert bool((p["y"] == 7).all())
