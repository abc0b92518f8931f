"""Host-side checks of the decode-step calls (include/lora_kv.h, include/lora_w4.h): sizes,
shapes and arguments are refused before anything is launched.  No GPU is used."""
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


def test_block_bytes():
    # 16 tokens of a head: 8 bytes a value of K and V together, and 8 bytes a group
    assert lora.kv_block_bytes(16, 1, 128, 128) == 16 * (128 + 8)
    assert lora.kv_block_bytes(64, 8, 128, 32) == 4 * 8 * 16 * (128 + 32)
    assert lora.kv_block_bytes(48, 3, 64, 64) == 3 * 3 * 16 * (64 + 8)
    for bad in ((8, 1, 128, 128), (0, 1, 128, 128), (16, 0, 128, 128), (16, 1, 96, 96), (16, 1, 128, 64), (16, 1, 64, 128)):
        assert status(lora.kv_block_bytes, *bad) == B.LORA_EINVAL, bad
    assert status(lora.kv_block_bytes, 1040, 1, 128, 128) == B.LORA_ETOOBIG
    assert status(lora.kv_block_bytes, 16, lora.LORA_KV_MAX_HEADS + 1, 128, 128) == B.LORA_ETOOBIG


def cache(**kw):
    d = dict(blocks=FAKE, num_blocks=10, block_stride=lora.kv_block_bytes(16, 2, 128, 128), block_tokens=16, num_kv_heads=2,
             head_dim=128, group=128)
    d.update(kw)
    return lora.KvCache(*d.values())


def batch(**kw):
    d = dict(q_start=FAKE, kv_len=FAKE, block_table=FAKE, n_seq=2, T=3, max_blocks=4, max_q=2)
    d.update(kw)
    return lora.KvBatch(*d.values())


def attend(kv=None, b=None, q=FAKE, ldq=512, heads=4, scale=0.1, out=FAKE, ldo=512, ws=FAKE, size=None):
    kv, b = kv or cache(), b or batch()
    size = lora.kv_workspace_size(cache(), batch(), 4) if size is None else size
    return status(lora.kv_attend, kv, b, q, ldq, heads, scale, out, ldo, None, ws, size, None)


def test_workspace_does_not_depend_on_the_batch():
    a = lora.kv_workspace_size(cache(), batch(), 4)
    assert a == lora.kv_workspace_size(cache(), batch(n_seq=500, T=4000, max_q=600), 4) and a % 256 == 0
    assert status(lora.kv_workspace_size, cache(), batch(), 3) == B.LORA_EINVAL
    assert status(lora.kv_workspace_size, cache(), batch(n_seq=-1), 4) == B.LORA_EINVAL
    assert status(lora.kv_workspace_size, cache(), batch(n_seq=lora.LORA_KV_MAX_SEQS + 1), 4) == B.LORA_ETOOBIG


def test_attention_refusals():
    assert attend(kv=cache(blocks=None)) == B.LORA_EINVAL
    assert attend(kv=cache(blocks=FAKE + 8)) == B.LORA_EALIGN
    assert attend(kv=cache(block_stride=lora.kv_block_bytes(16, 2, 128, 128) - 16)) == B.LORA_EINVAL
    assert attend(kv=cache(block_stride=lora.kv_block_bytes(16, 2, 128, 128) + 8)) == B.LORA_EALIGN
    assert attend(kv=cache(num_blocks=0)) == B.LORA_EINVAL
    assert attend(kv=cache(group=64)) == B.LORA_EINVAL
    assert attend(b=batch(kv_len=None)) == B.LORA_EINVAL
    assert attend(b=batch(T=-1)) == B.LORA_EINVAL
    assert attend(heads=3) == B.LORA_EINVAL
    assert attend(heads=0) == B.LORA_EINVAL
    assert attend(scale=0.0) == B.LORA_EINVAL
    assert attend(scale=float("inf")) == B.LORA_EINVAL
    assert attend(q=None) == B.LORA_EINVAL
    assert attend(q=FAKE + 2) == B.LORA_EALIGN
    assert attend(ldq=504) == B.LORA_EINVAL
    assert attend(ldo=516) == B.LORA_EALIGN
    assert attend(ws=None) == B.LORA_EWORKSPACE
    assert attend(ws=FAKE + 128) == B.LORA_EWORKSPACE
    assert attend(size=4096) == B.LORA_EWORKSPACE
    assert lora.lib().lora_kv_attend(None, None, None, 0, 4, 0.1, None, 0, None, None, 0, None) == B.LORA_EINVAL


def test_append_and_read_refusals():
    rope = lora.Rope(FAKE, FAKE, 100, 128)

    def append(rope=rope, q=FAKE, ldq=512, out=FAKE + 4096, ldqo=512, heads=4, k=FAKE, ldk=256, v=FAKE, ldv=256):
        return status(lora.kv_append, cache(), batch(), q, ldq, out, ldqo, heads, k, ldk, v, ldv, rope, FAKE, 4096, None)

    assert append(rope=lora.Rope(None, FAKE, 100, 128)) == B.LORA_EINVAL
    assert append(rope=lora.Rope(FAKE + 4, FAKE, 100, 128)) == B.LORA_EALIGN
    assert append(rope=lora.Rope(FAKE, FAKE, 0, 128)) == B.LORA_EINVAL
    assert append(rope=lora.Rope(FAKE, FAKE, 100, 144)) == B.LORA_EINVAL
    assert append(rope=lora.Rope(FAKE, FAKE, 100, 40)) == B.LORA_EINVAL
    assert append(rope=lora.Rope(FAKE, FAKE, 100, 128, 2)) == B.LORA_EINVAL
    assert append(heads=-1) == B.LORA_EINVAL
    assert append(q=None) == B.LORA_EINVAL
    assert append(out=FAKE, ldqo=520) == B.LORA_EINVAL          # in place with another pitch
    assert append(k=None) == B.LORA_EINVAL
    assert append(ldv=250) == B.LORA_EINVAL
    assert append(v=FAKE + 8) == B.LORA_EALIGN
    assert status(lora.kv_read, cache(), batch(), None, 256, FAKE, 256, FAKE, 4096, None) == B.LORA_EINVAL
    assert status(lora.kv_read, cache(), batch(), FAKE, 256, FAKE, 260, FAKE, 4096, None) == B.LORA_EALIGN
    assert status(lora.kv_read, cache(), batch(), FAKE, 256, FAKE, 256, FAKE, 128, None) == B.LORA_EWORKSPACE
    assert status(lora.kv_workspace_init, FAKE + 16, 4096, None) == B.LORA_EWORKSPACE
    assert status(lora.kv_workspace_init, FAKE, 100, None) == B.LORA_EWORKSPACE


def test_w4_refusals():
    def call(T=4, n=1, ws=FAKE, size=1 << 30, **kw):
        d = dict(x=FAKE, y=FAKE, ldx=256, ldy=64, codes=FAKE, scales=FAKE, zeros=FAKE, N=64, K=256, group=64)
        d.update(kw)
        return status(lora.w4_matvec, lora.w4_problems([tuple(d.values())] * n), T, ws, size, None)

    assert call(T=-1) == B.LORA_EINVAL
    assert call(T=lora.LORA_W4_MAX_ROWS + 1) == B.LORA_ETOOBIG
    assert call(n=lora.LORA_W4_MAX_PROBLEMS + 1) == B.LORA_ETOOBIG
    assert call(N=0) == B.LORA_EINVAL
    assert call(N=68) == B.LORA_EINVAL
    assert call(K=224) == B.LORA_EINVAL
    assert call(group=16) == B.LORA_EINVAL
    assert call(codes=None) == B.LORA_EINVAL
    assert call(scales=FAKE + 2) == B.LORA_EALIGN
    assert call(zeros=FAKE + 2) == B.LORA_EALIGN
    assert call(ldx=264 + 4) == B.LORA_EALIGN
    assert call(ldy=56) == B.LORA_EINVAL
    assert call(ws=None) == B.LORA_EWORKSPACE
    assert call(size=4096) == B.LORA_EWORKSPACE
    empty = lora.w4_problems([])
    lora.w4_matvec(empty, 4, None, 0, None)                    # nothing to do
    n = ctypes.c_size_t()
    assert lora.lib().lora_w4_workspace_size(None, 1, 4, ctypes.byref(n)) == B.LORA_EINVAL
    assert lora.lib().lora_w4_workspace_size(empty.ref, 0, 4, None) == B.LORA_EINVAL
