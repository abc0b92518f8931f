"""Rows left in 8 bits (include/lora_w8.h): the norm with the residual's addition and the gated
activation, against their definitions in 64 bits."""
import pytest

import heterogeneous_adapters_gb300 as lora

pytestmark = pytest.mark.gpu

WIDTHS = [16, 48, 64, 272, 1024, 4096, 4112, 5120, 8192, 14336, 16400, 32768]
ACTS = {"none": lora.LORA_ACT_NONE, "silu": lora.LORA_ACT_SILU, "gelu": lora.LORA_ACT_GELU, "gelu-tanh": lora.LORA_ACT_GELU_TANH}


def matrix(torch, g, T, d, pad=0):
    """bf16 [T][d] with a pitch of d + pad."""
    return torch.randn(T, d + pad, generator=g, device="cuda").bfloat16()[:, :d]


class Out:
    """Buffers for T rows, with two rows behind the last one and `pad` columns that stay as they are."""

    def __init__(self, torch, T, d, pad=0, kind=lora.LORA_Q8_X_HELD, x=True):
        self.T, self.d, self.kind = T, d, kind
        self.codes = torch.full((T + 2, d + 16 * (pad > 0)), 99, dtype=torch.int8, device="cuda")
        self.scales = torch.full((T + 2,), -3.0, device="cuda")
        self.x = torch.full((T + 2, d + pad), 7.0, dtype=torch.bfloat16, device="cuda") if x else None
        self.rows = lora.Q8Rows(self.codes, self.codes.stride(0), self.scales, self.x, d + pad if x else 0, kind)

    def untouched(self):
        T, d = self.T, self.d
        ok = bool((self.codes[T:] == 99).all()) and bool((self.codes[:, d:] == 99).all()) and bool((self.scales[T:] == -3).all())
        return ok and (self.x is None or bool((self.x[T:] == 7).all()) and bool((self.x[:, d:] == 7).all()))

    def got(self):
        return self.codes[:self.T, :self.d], self.scales[:self.T], None if self.x is None else self.x[:self.T, :self.d]


def stream(torch):
    return torch.cuda.current_stream().cuda_stream


def held(torch, codes, scales):
    """What codes stand for, in bf16: one fp32 product, rounded once."""
    return (codes.float() * scales[:, None]).bfloat16()


def run_norm(torch, x, residual, weight, eps=1e-5, kind=lora.LORA_Q8_X_HELD, pad=0, want_x=True, total=True):
    T, d = x.shape
    out = Out(torch, T, d, pad, kind, want_x)
    s = torch.full((T + 2, d + pad), 5.0, dtype=torch.bfloat16, device="cuda") if residual is not None and total else None
    call = lora.Q8Norm(x, x.stride(0), residual, residual.stride(0) if residual is not None else 0, s, d + pad, weight, eps, d, out.rows)
    lora.q8_norm(call, T, stream(torch))
    torch.cuda.synchronize()
    assert out.untouched() and (s is None or bool((s[T:] == 5).all()) and bool((s[:, d:] == 5).all()))
    return (*out.got(), None if s is None else s[:T, :d])


def check_norm(torch, x, residual, weight, eps=1e-5, kind=lora.LORA_Q8_X_HELD, **kw):
    codes, scales, xo, total = run_norm(torch, x, residual, weight, eps, kind, **kw)
    h = x.float()
    if residual is not None:
        h = (h + residual.float()).bfloat16().float()
        assert total is None or torch.equal(total.float(), h)
    h = h.double()
    p = h * weight.double()                                   # exact: products of 8-bit mantissas
    top = p.abs().amax(1, keepdim=True)
    want = torch.round(127 * p / torch.where(top > 0, top, 1.0))
    assert torch.equal(codes.double(), want)
    over = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    scale = (top * over / 127)[:, 0]
    # a thread adds at most 32 squares, ten steps join the threads: 42 roundings of 2^-24 of the sum,
    # half of that after the root, and six more roundings: 27 * 2^-24
    assert bool(((scales.double() - scale).abs() <= 27 * 2.0 ** -24 * scale).all())
    if xo is not None and kind == lora.LORA_Q8_X_HELD:
        assert torch.equal(xo, held(torch, codes, scales))
    elif xo is not None:
        y = p * over
        assert bool(((xo.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -18) * y.abs()).all())


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("T", [1, 2, 5, 130])
@pytest.mark.parametrize("add", [True, False])
def test_norm(cuda, d, T, add):
    g = cuda.Generator(device="cuda").manual_seed(d + T)
    pad = 8 * (T % 3)
    x, r = matrix(cuda, g, T, d, pad), matrix(cuda, g, T, d, 2 * pad) * 3 if add else None
    w = (1 + 0.2 * cuda.randn(d, generator=g, device="cuda")).bfloat16()
    check_norm(cuda, x, r, w, pad=pad, kind=lora.LORA_Q8_X_FULL if T == 5 else lora.LORA_Q8_X_HELD, want_x=T != 2, total=T != 5)


def test_norm_many_rows(cuda):
    g = cuda.Generator(device="cuda").manual_seed(3)
    for T, d in ((5001, 4096), (3000, 64), (1111, 1040)):
        x, r = matrix(cuda, g, T, d), matrix(cuda, g, T, d)
        check_norm(cuda, x, r, (1 + 0.2 * cuda.randn(d, generator=g, device="cuda")).bfloat16())


def test_quotients_on_a_half(cuda):
    """Codes whose quotients lie on a half go to the even one, whatever the largest value is."""
    d = 512
    k = cuda.arange(d, device="cuda") % 255 - 127
    x = k.bfloat16()[None].repeat(6, 1)                       # whole numbers up to 127, exact in bf16
    x[0, 0], x[1, 0], x[2, 0] = 254, 254, 127                 # quotients k / 2, k / 2 and k
    x[3, 0], x[4, 0], x[5, 0] = 508 / 2, -254, 250
    w = cuda.ones(d, device="cuda").bfloat16()
    check_norm(cuda, x, None, w)
    w = (2.0 ** cuda.randint(-3, 3, (d,), device="cuda").float()).bfloat16()
    check_norm(cuda, x, None, w)
    w = cuda.full((d,), 1.5, device="cuda").bfloat16()
    w[::3] = 0.75
    check_norm(cuda, x, x, w)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-10, 1e10, 1e18, 3e19, 1e30, 1e38])
def test_norm_sizes(cuda, size):
    """Rows whose squares leave fp32's range: scales and codes as in 64 bits."""
    g = cuda.Generator(device="cuda").manual_seed(1)
    x = (cuda.randn(4, 4096, generator=g, device="cuda").clamp(-3, 3) * size).bfloat16()
    x[1] *= 0.25
    w = (1 + 0.2 * cuda.randn(4096, generator=g, device="cuda").clamp(-3, 3)).bfloat16()
    if size <= 1e-38:
        x *= 2.0 ** 10
    check_norm(cuda, x, None, w, eps=1e-30 if size == 1e-10 else 1e-5)
    check_norm(cuda, x, None, w, kind=lora.LORA_Q8_X_FULL)


def test_norm_rows_of_zeros_and_without_a_number(cuda):
    g = cuda.Generator(device="cuda").manual_seed(2)
    x = matrix(cuda, g, 9, 1024)
    clean = x.clone()
    x[1] = 0
    x[3, 7] = float("inf")
    x[4, 1000] = float("nan")
    x[6, 0] = -float("inf")
    w = (1 + 0.2 * cuda.randn(1024, generator=g, device="cuda")).bfloat16()
    w[1000] = 0                                               # not a number at any weight
    for kind in (lora.LORA_Q8_X_HELD, lora.LORA_Q8_X_FULL):
        codes, scales, xo, _ = run_norm(cuda, x, None, w, kind=kind)
        for t in (3, 4, 6):
            assert bool(scales[t].isnan()) and not bool(codes[t].any()) and bool(xo[t].isnan().all())
        assert float(scales[1]) == 0 and not bool(codes[1].any()) and not bool(xo[1].any())
        c2, s2, x2, _ = run_norm(cuda, clean, None, w, kind=kind)
        rest = [0, 2, 5, 7, 8]
        assert cuda.equal(codes[rest], c2[rest]) and cuda.equal(scales[rest], s2[rest]) and cuda.equal(xo[rest], x2[rest])


@pytest.mark.parametrize("d", [64, 4096, 16384])
def test_norm_in_place(cuda, d):
    """The sum in the place of x or of the residual."""
    g = cuda.Generator(device="cuda").manual_seed(d)
    x, r = matrix(cuda, g, 33, d), matrix(cuda, g, 33, d)
    w = (1 + 0.2 * cuda.randn(d, generator=g, device="cuda")).bfloat16()
    codes, scales, xo, total = run_norm(cuda, x, r, w)
    for which in (0, 1):
        a = [x.clone(), r.clone()]
        out = Out(cuda, 33, d)
        lora.q8_norm(lora.Q8Norm(a[0], d, a[1], d, a[which], d, w, 1e-5, d, out.rows), 33, stream(cuda))
        assert cuda.equal(a[which], total) and cuda.equal(a[1 - which], (x, r)[1 - which])
        assert all(cuda.equal(p, q) for p, q in zip(out.got(), (codes, scales, xo)))


def activation(torch, name, a):
    if name == "silu":
        return a * torch.sigmoid(a)
    if name == "gelu":
        return a * torch.special.ndtr(a)
    if name == "gelu-tanh":
        return a * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (a + 0.044715 * a ** 3))
    return a


def run_gate(torch, gate, up, act, kind=lora.LORA_Q8_X_HELD, pad=0, want_x=True):
    T, d = gate.shape
    out = Out(torch, T, d, pad, kind, want_x)
    call = lora.Q8Gate(gate, gate.stride(0), up, up.stride(0) if up is not None else 0, ACTS[act], d, out.rows)
    lora.q8_gate(call, T, stream(torch))
    torch.cuda.synchronize()
    assert out.untouched()
    return out.got()


def check_gate(torch, gate, up, act, kind=lora.LORA_Q8_X_HELD, **kw):
    codes, scales, xo = run_gate(torch, gate, up, act, kind, **kw)
    y = activation(torch, act, gate.double())
    size = gate.double().abs()                                # 1 + erf and 1 + tanh are rounded at their size, not at their sum's
    if up is not None:
        y, size = y * up.double(), size * up.double().abs()
    # an exponential of a rounded argument up to 90, a sum, a quotient and two products: 90 + 10 roundings of 2^-24
    tol = 100 * 2.0 ** -24 * y.abs() + 4 * 2.0 ** -24 * size if act != "none" else 2.0 ** -24 * y.abs()
    top, at = y.abs().max(1)
    slack = tol.gather(1, at[:, None])[:, 0] + tol.amax(1)
    assert bool(((scales.double() * 127 - top).abs() <= 3 * 2.0 ** -24 * top + slack).all())
    assert bool((codes.abs().amax(1) == 127)[top > 0].all())
    step = scales.double()[:, None]
    # half a step, and 127 roundings of its size
    assert bool(((codes.double() * step - y).abs() <= (0.5 + 127 * 4 * 2.0 ** -24) * step + tol).all())
    if xo is not None and kind == lora.LORA_Q8_X_HELD:
        assert torch.equal(xo, held(torch, codes, scales))
    elif xo is not None:
        assert bool(((xo.double() - y).abs() <= 2.0 ** -8 * (y.abs() + tol) + tol).all())
    if act == "none" and up is None:
        g = gate.double()
        assert torch.equal(codes.double(), torch.round(127 * g / torch.where(top > 0, top, 1.0)[:, None]))


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("gated", [True, False])
def test_gate(cuda, d, act, gated):
    g = cuda.Generator(device="cuda").manual_seed(d)
    for T in (1, 3, 66):
        pad = 8 * (T % 3)
        both = matrix(cuda, g, T, 2 * d, pad) * 2
        check_gate(cuda, both[:, :d], both[:, d:2 * d] if gated else None, act, pad=pad,
                   kind=lora.LORA_Q8_X_FULL if T == 3 else lora.LORA_Q8_X_HELD, want_x=T != 1)


def test_gate_many_rows(cuda):
    g = cuda.Generator(device="cuda").manual_seed(3)
    for T, d in ((2001, 14336), (4000, 112)):
        both = matrix(cuda, g, T, 2 * d)
        check_gate(cuda, both[:, :d], both[:, d:], "silu")


@pytest.mark.parametrize("size", [1e-35, 1e-30, 1e-19, 1e-8, 1e8, 1e30])
def test_gate_sizes(cuda, size):
    g = cuda.Generator(device="cuda").manual_seed(1)
    a = (cuda.randn(4, 512, generator=g, device="cuda") * size).bfloat16()
    one = cuda.ones_like(a)
    check_gate(cuda, a, None, "none")
    check_gate(cuda, a, one, "none")
    if size < 1e20:
        check_gate(cuda, one, a, "silu")
    if size > 1:
        for act in ("silu", "gelu", "gelu-tanh"):             # each value is itself or nothing
            check_gate(cuda, a, one, act)


def test_gate_rows_of_zeros_and_without_a_number(cuda):
    g = cuda.Generator(device="cuda").manual_seed(2)
    a, u = matrix(cuda, g, 8, 1024), matrix(cuda, g, 8, 1024)
    a[1] = 0
    a[2, 5] = -float("inf")                                   # an activation of nothing, but not of a number
    u[3, 9] = float("nan")
    u[4, 9] = float("inf")
    a[4, 9] = 0
    a[6, 1] = float("nan")
    for act in ACTS:
        codes, scales, xo = run_gate(cuda, a, u, act)
        for t in (2, 3, 4, 6):
            assert bool(scales[t].isnan()) and not bool(codes[t].any()) and bool(xo[t].isnan().all()), (act, t)
        assert float(scales[1]) == 0 and not bool(codes[1].any()) and not bool(xo[1].any())
        check_gate(cuda, a[[0, 5, 7]], u[[0, 5, 7]], act)


def test_gate_in_place(cuda):
    """x in the place of the gate or of the other factor."""
    g = cuda.Generator(device="cuda").manual_seed(5)
    for d in (64, 14336):
        a, u = matrix(cuda, g, 17, d), matrix(cuda, g, 17, d)
        want = run_gate(cuda, a, u, "silu")
        for which in (0, 1):
            b = [a.clone(), u.clone()]
            codes, scales = cuda.empty(17, d, dtype=cuda.int8, device="cuda"), cuda.empty(17, device="cuda")
            rows = lora.Q8Rows(codes, d, scales, b[which], d)
            lora.q8_gate(lora.Q8Gate(b[0], d, b[1], d, lora.LORA_ACT_SILU, d, rows), 17, stream(cuda))
            assert cuda.equal(codes, want[0]) and cuda.equal(scales, want[1]) and cuda.equal(b[which], want[2])


def test_no_rows(cuda):
    x = cuda.zeros(4, 64, dtype=cuda.bfloat16, device="cuda")
    out = Out(cuda, 0, 64)
    lora.q8_norm(lora.Q8Norm(x, 64, None, 0, None, 0, x, 1e-5, 64, out.rows), 0, stream(cuda))
    lora.q8_gate(lora.Q8Gate(x, 64, None, 0, lora.LORA_ACT_NONE, 64, out.rows), 0, stream(cuda))
    assert out.untouched()


def test_in_place_with_more_rows_than_the_device_holds(cuda):
    """A CTA's next row is fetched before the one before it is written."""
    g = cuda.Generator(device="cuda").manual_seed(6)
    for T, d in ((3001, 64), (1203, 4096), (701, 4112)):
        x, r = matrix(cuda, g, T, d), matrix(cuda, g, T, d)
        w = (1 + 0.2 * cuda.randn(d, generator=g, device="cuda")).bfloat16()
        codes, scales, xo, total = run_norm(cuda, x, r, w)
        out = Out(cuda, T, d)
        lora.q8_norm(lora.Q8Norm(x, d, r, d, x, d, w, 1e-5, d, out.rows), T, stream(cuda))
        assert cuda.equal(x, total) and all(cuda.equal(p, q) for p, q in zip(out.got(), (codes, scales, xo)))
        want = run_gate(cuda, x, r, "silu")
        rows = lora.Q8Rows(out.codes, out.codes.stride(0), out.scales, r, d)
        lora.q8_gate(lora.Q8Gate(x, d, r, d, lora.LORA_ACT_SILU, d, rows), T, stream(cuda))
        assert cuda.equal(out.codes[:T], want[0]) and cuda.equal(out.scales[:T], want[1]) and cuda.equal(r, want[2])
