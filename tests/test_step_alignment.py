"""Host-side refusals of misaligned arrays of 32-bit values (include/lora_kv.h).  No GPU is used."""
import pytest

import heterogeneous_adapters_gb300 as lora
from heterogeneous_adapters_gb300 import _binding as B

from .test_step_abi import FAKE, batch, built, cache, status  # noqa: F401

WS = (FAKE, 1 << 30, None)


@pytest.mark.parametrize("name", ["q_start", "kv_len", "block_table"])
@pytest.mark.parametrize("by", [1, 2])
def test_batch_arrays(name, by):
    b, rope = batch(**{name: FAKE + by}), lora.Rope(None, None, 0, 0)
    assert status(lora.kv_attend, cache(), b, FAKE, 512, 4, 0.1, FAKE, 512, None, *WS) == B.LORA_EALIGN
    assert status(lora.kv_read, cache(), b, FAKE, 256, FAKE, 256, *WS) == B.LORA_EALIGN
    assert status(lora.kv_append, cache(), b, None, 0, None, 0, 0, FAKE, 256, FAKE, 256, rope, *WS) == B.LORA_EALIGN


@pytest.mark.parametrize("by", [1, 2])
def test_positions_and_log_sums(by):
    rope = lora.Rope(FAKE, FAKE, 100, 64, positions=FAKE + by)
    assert status(lora.kv_append, cache(), batch(), None, 0, None, 0, 0, FAKE, 256, FAKE, 256, rope, *WS) == B.LORA_EALIGN
    assert status(lora.kv_attend, cache(), batch(), FAKE, 512, 4, 0.1, FAKE, 512, FAKE + by, *WS) == B.LORA_EALIGN
