"""Linear attention where one value's reach is the question.  What must not reach an
output must not change one bit of it; values are held to the tolerances of
test_gpu_linear_attention."""
import pytest
import torch

import selective_state_update_gb300 as ssu
from test_gpu_linear_attention import DEV, check_prefill, problem

pytestmark = pytest.mark.gpu


def fill_tensor_memory(dstate, heads=320):
    """Leaves finite growths near 1e32 in the tensor memory of every SM (more heads than SMs)."""
    big = torch.full((1, heads, 128, dstate), 0.0, device=DEV)
    x = torch.full((128, heads, 128), 2.0 ** 50, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 128], dtype=torch.int32, device=DEV)
    ssu.ssu_linear_attention_prefill(big, x[..., :dstate], x[..., :dstate], x, torch.zeros(heads, device=DEV), cu)
    assert 1e31 < float(big.max()) < 1e33


@pytest.mark.parametrize("before,dstate", [(128, 96), (128, 72), (128, 112), (64, 32), (64, 8), (128, 48)])
def test_prefill_fp16_after_large_growths(libssu, before, dstate):
    """Nothing of an earlier call is left in what the state's rows are scaled by."""
    fill_tensor_memory(before)
    check_prefill(200 + dstate, [300, 131], 80, 80, 64, dstate, torch.float16, torch.float32)
