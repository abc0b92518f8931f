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
