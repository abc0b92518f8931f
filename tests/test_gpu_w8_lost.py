"""The self-test of the wide products' waits (include/lora_w8.h) at the call's last step and past it."""
import pytest

import heterogeneous_adapters_gb300 as lora
from heterogeneous_adapters_gb300 import _binding as B

from .test_gpu_w8 import check, problem, problems, workspace

pytestmark = pytest.mark.gpu


# one tile along x each, 256 rows of W and 128 of K a step
@pytest.mark.parametrize("T,N,K,most", [(40, 8192, 4096, 32 * 32), (64, 14336, 4096, 56 * 32), (33, 32776, 400, 129 * 4)])
def test_a_step_past_the_last_is_refused(cuda, T, N, K, most):
    g = cuda.Generator(device="cuda").manual_seed(T)
    p = problem(cuda, g, T, N, K)
    pr = problems([p])
    ws, size = workspace(cuda, pr, T)
    stream = cuda.cuda.current_stream().cuda_stream
    for step in (most, most + 1, 2 ** 31 - 1):
        with pytest.raises(lora.LoraError) as e:
            lora.debug_w8_lost_step(pr, T, step, 5_000_000, ws, size, stream)
        assert e.value.status == B.LORA_EINVAL
    assert bool((p["y"] == 7).all()) and lora.get_device_error(ws, stream) == 0
    lora.debug_w8_lost_step(pr, T, most - 1, 5_000_000, ws, size, stream)
    assert lora.get_device_error(ws, stream) == 0x20
    lora.w8_matmul(pr, T, ws, size, stream)
    assert lora.get_device_error(ws, stream) == 0
    check(cuda, p)
