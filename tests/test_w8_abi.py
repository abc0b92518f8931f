"""Host-side checks of an 8-bit base model's calls (include/lora_w8.h): sizes, shapes and
arguments are refused before anything is launched.  No GPU is used."""
import ctypes

import pytest

import heterogeneous_adapters_gb300 as lora
from heterogeneous_adapters_gb300 import _binding as B

FAKE = 1 << 20      # an address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    from heterogeneous_adapters_gb300 import build
    build.build()


def status(f, *a):
    with pytest.raises(lora.LoraError) as e:
        f(*a)
    return e.value.status


def rows(**kw):
    d = dict(codes=FAKE, ldc=64, scales=FAKE, x=FAKE, ldx=64, x_kind=lora.LORA_Q8_X_HELD)
    d.update(kw)
    return lora.Q8Rows(*d.values())


BAD_ROWS = [(dict(codes=None), B.LORA_EINVAL), (dict(scales=None), B.LORA_EINVAL), (dict(codes=FAKE + 8), B.LORA_EALIGN),
            (dict(ldc=72), B.LORA_EALIGN), (dict(ldc=48), B.LORA_EINVAL), (dict(scales=FAKE + 2), B.LORA_EALIGN),
            (dict(x=FAKE + 2), B.LORA_EALIGN), (dict(ldx=68), B.LORA_EALIGN), (dict(ldx=56), B.LORA_EINVAL),
            (dict(x_kind=2), B.LORA_EINVAL), (dict(x_kind=-1), B.LORA_EINVAL)]


def norm(T=4, out=None, **kw):
    d = dict(x=FAKE, ldx=64, residual=FAKE, ldr=64, total=FAKE + 4096, lds=64, weight=FAKE, eps=1e-5, d=64)
    d.update(kw)
    return status(lora.q8_norm, lora.Q8Norm(*d.values(), out or rows()), T, None)


def test_norm_refusals():
    assert norm(T=-1) == B.LORA_EINVAL
    assert norm(T=lora.LORA_Q8_MAX_ROWS + 1) == B.LORA_ETOOBIG
    assert norm(d=0) == B.LORA_EINVAL
    assert norm(d=-16) == B.LORA_EINVAL
    assert norm(d=56) == B.LORA_EINVAL
    big = lora.LORA_Q8_MAX_WIDTH + 16
    assert norm(d=big, ldx=big) == B.LORA_ETOOBIG
    for eps in (0.0, -1e-5, 1e-31, float("nan"), float("inf")):
        assert norm(eps=eps) == B.LORA_EINVAL, eps
    assert norm(x=None) == B.LORA_EINVAL
    assert norm(x=FAKE + 4) == B.LORA_EALIGN
    assert norm(ldx=56) == B.LORA_EINVAL
    assert norm(ldx=68) == B.LORA_EALIGN
    assert norm(residual=FAKE + 8) == B.LORA_EALIGN
    assert norm(ldr=48) == B.LORA_EINVAL
    assert norm(residual=None) == B.LORA_EINVAL                 # a sum of nothing
    assert norm(total=FAKE + 2) == B.LORA_EALIGN
    assert norm(lds=32) == B.LORA_EINVAL
    assert norm(total=FAKE, lds=72) == B.LORA_EINVAL            # in place with another pitch
    assert norm(weight=None) == B.LORA_EINVAL
    assert norm(weight=FAKE + 2) == B.LORA_EALIGN
    for kw, want in BAD_ROWS:
        assert norm(out=rows(**kw)) == want, kw
    bad = rows()
    bad.struct.reserved = 1
    assert norm(out=bad) == B.LORA_EINVAL
    assert lora.lib().lora_q8_norm(None, 4, None) == B.LORA_EINVAL


def gate(T=4, out=None, **kw):
    d = dict(gate=FAKE, ldg=128, up=FAKE + 128, ldu=128, act=lora.LORA_ACT_SILU, d=64)
    d.update(kw)
    return status(lora.q8_gate, lora.Q8Gate(*d.values(), out or rows()), T, None)


def test_gate_refusals():
    assert gate(T=-1) == B.LORA_EINVAL
    assert gate(T=lora.LORA_Q8_MAX_ROWS + 1) == B.LORA_ETOOBIG
    assert gate(d=24) == B.LORA_EINVAL
    assert gate(act=4) == B.LORA_EINVAL
    assert gate(act=-1) == B.LORA_EINVAL
    assert gate(gate=None) == B.LORA_EINVAL
    assert gate(gate=FAKE + 2) == B.LORA_EALIGN
    assert gate(ldg=32) == B.LORA_EINVAL
    assert gate(up=FAKE + 8) == B.LORA_EALIGN
    assert gate(ldu=60) == B.LORA_EALIGN
    assert gate(out=rows(x=FAKE + 128)) == B.LORA_EINVAL        # in place with another pitch
    for kw, want in BAD_ROWS:
        assert gate(out=rows(**kw)) == want, kw
    assert lora.lib().lora_q8_gate(None, 4, None) == B.LORA_EINVAL


def problem(**kw):
    d = dict(x=FAKE, x_scales=FAKE, y=FAKE, ldx=256, ldy=64, w=FAKE, w_scales=FAKE, N=64, K=256)
    d.update(kw)
    return tuple(d.values())


def test_product_refusals():
    def call(T=4, n=1, ws=FAKE, size=1 << 40, **kw):
        return status(lora.w8_matmul, lora.w8_problems([problem(**kw)] * n), T, ws, size, None)

    assert call(T=-1) == B.LORA_EINVAL
    assert call(T=lora.LORA_W8_MAX_ROWS + 1) == B.LORA_ETOOBIG
    assert call(n=lora.LORA_W8_MAX_PROBLEMS + 1) == B.LORA_ETOOBIG
    assert call(N=0) == B.LORA_EINVAL
    assert call(N=68) == B.LORA_EINVAL
    assert call(N=(1 << 24) + 8) == B.LORA_ETOOBIG
    assert call(K=0) == B.LORA_EINVAL
    assert call(K=200) == B.LORA_EINVAL
    assert call(K=lora.LORA_W8_MAX_K + 16) == B.LORA_ETOOBIG
    for name in ("x", "x_scales", "y", "w", "w_scales"):
        assert call(**{name: None}) == B.LORA_EINVAL, name
        assert call(**{name: FAKE + 2}) == B.LORA_EALIGN, name
    assert call(ldx=240) == B.LORA_EINVAL
    assert call(ldx=264) == B.LORA_EALIGN
    assert call(ldy=56) == B.LORA_EINVAL
    assert call(ldy=68) == B.LORA_EALIGN
    assert call(ws=None) == B.LORA_EWORKSPACE
    assert call(ws=FAKE + 128) == B.LORA_EWORKSPACE
    assert call(size=256) == B.LORA_EWORKSPACE
    lora.w8_matmul(lora.w8_problems([]), 4, None, 0, None)      # nothing to do
    n = ctypes.c_size_t()
    assert lora.lib().lora_w8_workspace_size(None, 1, 4, ctypes.byref(n)) == B.LORA_EINVAL
    assert lora.lib().lora_w8_workspace_size(lora.w8_problems([problem()]).ref, 1, 4, None) == B.LORA_EINVAL


def test_workspace_grows_with_the_rows():
    """A workspace for T rows serves every call of fewer, and shared rows are counted once."""
    shared = [problem(), problem(N=128, ldy=128)]
    apart = [problem(), problem(N=128, ldy=128, x=2 * FAKE)]
    last = 0
    for T in (0, 1, 8, 9, 16, 31, 32, 33, 64, 65, 200, 256, 257, 1000, 4097, lora.LORA_W8_MAX_ROWS):
        a, b = (lora.w8_workspace_size(lora.w8_problems(p), T) for p in (shared, apart))
        assert a % 256 == 0 and last <= a <= b
        last = a
    assert status(lora.w8_workspace_size, lora.w8_problems(shared), -1) == B.LORA_EINVAL
