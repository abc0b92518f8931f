"""Rows left in 8 bits (include/lora_w8.h) at the ends of their operators' ranges: activations far below
zero, norms of rows whose squares or products leave fp32's range."""
import pytest

import heterogeneous_adapters_gb300 as lora

from .test_gpu_q8 import activation, held, matrix, run_gate

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                                # half a step of fp32


def value(torch, act, a):
    """act(a) in 64 bits (erfc: 1 + erf has no digits left in 64 bits either below -8)."""
    return 0.5 * a * torch.special.erfc(-a * 0.5 ** 0.5) if act == "gelu" else activation(torch, act, a)


def roundings(torch, act, a):
    """Roundings of 2^-24 between gate a and act(a), each relative to act(a).  Every form has an exponential to 2 ulp (4), of
    an argument whose error it takes over in full: its roundings times its size."""
    if act == "silu":
        # argument: a constant (half a rounding) and a product; the exponential; a sum, a quotient to 1 ulp, a product
        return 1.5 * a.abs() + 10
    if act == "gelu-tanh":
        # argument 2 (2 / pi)^1/2 (a + 0.044715 a^3): constants, a square, a sum and two products, six in all
        return 6 * (2 * (2 / torch.pi) ** 0.5 * (a.abs() + 0.044715 * a.abs() ** 3)) + 10
    # argument a^2 / 2: a constant and a product; F: 7, two products more and the difference
    return 0.75 * a ** 2 + 16


def check_close(torch, gate, up, act, kind=lora.LORA_Q8_X_HELD):
    """Every value to a share of its own size, however small it is beside the gate."""
    codes, scales, xo = run_gate(torch, gate, up, act, kind)
    y = value(torch, act, gate.double())
    tol = (roundings(torch, act, gate.double()) + 1) * U      # and the product with up
    # below the smallest normal value, 2^-126, an activation may be nothing, and so may y's digits (bf16's steps are 2^-133 there)
    least = torch.full_like(y, 2.0 ** -126)
    if up is not None:
        y, least = y * up.double(), least * up.double().abs().clamp(min=1)
    tol = tol * y.abs() + least
    top, at = y.abs().max(1)
    slack = tol.gather(1, at[:, None])[:, 0]
    assert bool(((scales.double() * 127 - top).abs() <= 3 * U * top + torch.maximum(slack, tol.amax(1))).all())
    assert bool((codes.abs().amax(1) == 127).all())
    step = scales.double()[:, None]
    assert bool(((codes.double() * step - y).abs() <= (0.5 + 127 * 4 * U) * step + tol).all())
    if kind == lora.LORA_Q8_X_HELD:
        assert torch.equal(xo, held(torch, codes, scales))
    else:
        assert bool(((xo.double() - y).abs() <= 2.0 ** -8 * (y.abs() + tol) + tol).all())


@pytest.mark.parametrize("act,low,high", [("gelu", -13, -9), ("gelu", -9, -4), ("gelu", -5.5, 0), ("gelu", -4, 4), ("gelu", 0, 14),
                                          ("silu", -100, -70), ("silu", -86.75, -86.25), ("silu", -20, 10), ("silu", 80, 100),
                                          ("gelu-tanh", -10.5, -9), ("gelu-tanh", -9, -4), ("gelu-tanh", -4, 4), ("gelu-tanh", 4, 14)])
@pytest.mark.parametrize("large", [False, True])
def test_activations_keep_their_digits(cuda, act, low, high, large):
    """Rows of gates in a range, without up, with one of ordinary values and with large ones beside the lowest gates."""
    g = cuda.Generator(device="cuda").manual_seed(int(high) + 100)
    for T, d in ((3, 512), (40, 4096), (5, 16400)):
        gate = (low + (high - low) * cuda.rand(T, d, generator=g, device="cuda")).bfloat16()
        up = matrix(cuda, g, T, d)
        if large:
            up = (up.double() * (gate.double() < (low + high) / 2) * 2.0 ** 60 + up.double()).bfloat16()
        for kind in (lora.LORA_Q8_X_HELD, lora.LORA_Q8_X_FULL):
            check_close(cuda, gate, None, act, kind)
            check_close(cuda, gate, up, act, kind)


@pytest.mark.parametrize("act,gates", [("gelu", 20), ("silu", 128), ("gelu-tanh", 20)])
def test_every_gate(cuda, act, gates):
    """Rows of one gate, and of one gate beside zeros: all bf16 values of a size from 2^-30 to `gates` whose activation is
    a normal fp32 value, alone and with a factor that takes the smallest ones where 8 bits and bf16 hold them."""
    bits = cuda.arange((127 - 30) << 7, (127 + 7) << 7, device="cuda", dtype=cuda.int32)
    a = cuda.cat([bits, bits + 0x8000]).to(cuda.int16).view(cuda.bfloat16)
    a = a[a.abs() <= gates]
    size = value(cuda, act, a.double()).abs()
    for least, factor in ((2.0 ** -100, None), (2.0 ** -100, 2.0 ** -20), (2.0 ** -125, 2.0 ** 40), (2.0 ** -125, 2.0 ** 100)):
        rows = a[size > least][:, None].repeat(1, 32).contiguous()
        rows[1::2, 1:] = 0
        up = None if factor is None else cuda.full_like(rows, factor)
        check_close(cuda, rows, up, act)
        check_close(cuda, rows, up, act, lora.LORA_Q8_X_FULL)


def run_in(torch, x, residual, weight, eps, kind, place):
    """A norm with its sum in a place of its own, nowhere, or where x or the residual was."""
    T, d = x.shape
    a = [x.clone(), residual.clone()] if residual is not None else [x.clone(), None]
    total = {"own": torch.empty_like(x), "none": None, "x": a[0], "residual": a[1]}[place] if residual is not None else None
    codes, scales, xo = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
    lora.q8_norm(lora.Q8Norm(a[0], d, a[1], d, total, d, weight, eps, d, lora.Q8Rows(codes, d, scales, xo, d, kind)), T,
                 torch.cuda.current_stream().cuda_stream)
    return codes, scales, xo, total


def check_norm_range(torch, x, residual, weight, eps, place):
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    p = h.double() * weight.double()
    top = p.abs().amax(1, keepdim=True)
    over = 1 / torch.sqrt(h.double().square().mean(1, keepdim=True) + eps)
    y = p * over
    for kind in (lora.LORA_Q8_X_HELD, lora.LORA_Q8_X_FULL):
        codes, scales, xo, total = run_in(torch, x, residual, weight, eps, kind, place)
        assert total is None or torch.equal(total, h)
        assert torch.equal(codes.double(), torch.round(127 * p / torch.where(top > 0, top, 1.0)))
        want = (top * over / 127)[:, 0]
        # a thread adds at most 32 squares, ten steps join the threads: 42 roundings of 2^-24 of the sum, half of that after
        # the root, and six more roundings, the last one, by a power of two, of half a step of 2^-149 below the normal values
        assert bool(((scales.double() - want).abs() <= 27 * U * want + 2.0 ** -150).all())
        if kind == lora.LORA_Q8_X_HELD:
            assert torch.equal(xo, held(torch, codes, scales))
        else:
            # the smallest of a row may be nothing, and bf16's steps below its normal values are 2^-133
            assert bool(((xo.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -18) * y.abs() + 2.0 ** -64 * y.abs().amax(1, keepdim=True) + 2.0 ** -134).all())


# sizes of h and of the weights, eps, and what stands in channel 3 of a row: h and the weight
SIZES = [(1, 1e-30, 1e-5, None), (1, 1e-35, 1e-5, None), (1, 1e35, 1e-5, None), (1e-15, 1e20, 1e-30, None), (1e-20, 1e-15, 1e-30, None),
         (1e15, 1e30, 1e-5, None), (1e15, 1e-30, 1e-5, None), (1e18, 1e-10, 1e-5, None), (1e30, 1e-30, 1e-5, None), (1e30, 1e6, 1e-5, None),
         (1e25, 1e30, 1e-5, None), (1e30, 1e-2, 1e-5, None), (1, 2.0 ** -70, 1e-5, (2.0 ** 40, 0)), (1, 2.0 ** -100, 1e-5, (2.0 ** 40, 0)),
         (1, 2.0 ** -97, 1e-5, (2.0 ** 62, 2.0 ** -126)), (1, 1, 1e-5, (2.0 ** 60, 2.0 ** 45)), (1, 1e20, 1e-5, (2.0 ** 100, 0)),
         (2.0 ** -100, 2.0 ** 20, 1e-30, (2.0 ** -130, 2.0 ** 120))]


@pytest.mark.parametrize("place", ["alone", "own", "none", "x", "residual"])
@pytest.mark.parametrize("size,weight,eps,channel", SIZES)
def test_norms_near_the_ends_of_the_range(cuda, size, weight, eps, channel, place):
    """Squares and products of h and the weights far from 1, on either side or both: codes, scales and sums as in 64 bits."""
    g = cuda.Generator(device="cuda").manual_seed(8)
    for d in (512, 8192):
        x, r = ((cuda.randn(5, d, generator=g, device="cuda").clamp(-3, 3) * size).bfloat16() for _ in range(2))
        w = ((1 + 0.2 * cuda.randn(d, generator=g, device="cuda").clamp(-3, 3)) * weight).bfloat16()
        x[1] *= 0.25
        x[2], r[2] = 0, 0
        if channel is not None:
            x[::2, 3], r[::2, 3], w[3] = channel[0], 0, channel[1]
            x[2, 3] = 0
        check_norm_range(cuda, x, None if place == "alone" else r, w, eps, place)


def test_norms_without_a_number_near_the_ends(cuda):
    """Rows that are not finite where squares and products leave the range as well, and a scale that does."""
    x = cuda.full((6, 32768), 1.0, device="cuda").bfloat16()
    for big, weight in ((1.0, 1e-35), (1e30, 1.0), (1e30, 1e-35), (1e15, 1e30), (1e25, 1e30)):
        a = (x * big).bfloat16()
        a[1, 7], a[3, 30000], a[4, 0] = float("nan"), float("inf"), -float("inf")
        w = cuda.full((32768,), weight, device="cuda").bfloat16()
        codes, scales, xo, _ = run_in(cuda, a, None, w, 1e-5, lora.LORA_Q8_X_HELD, "none")
        for t in (1, 3, 4):
            assert bool(scales[t].isnan()) and not bool(codes[t].any()) and bool(xo[t].isnan().all())
        for t in (0, 2, 5):
            assert bool(scales[t].isfinite()) and bool((codes[t] == 127).all())
    one = cuda.zeros_like(x)
    one[:, 5] = 1
    one[2] = 1
    w = cuda.full((32768,), 3e38, device="cuda").bfloat16()
    codes, scales, xo, _ = run_in(cuda, one, None, w, 1e-5, lora.LORA_Q8_X_HELD, "none")   # y of 181 3e38: a 127th of it is too large
    for t in (0, 1, 3, 4, 5):
        assert bool(scales[t].isnan()) and not bool(codes[t].any())
    assert bool(scales[2].isfinite()) and bool((codes[2] == 127).all())
