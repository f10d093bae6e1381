"""Log probabilities of rows whose logits are large in size: the exponents are
taken against a rounded reference, whose rounding grows with them.  Held to the
tolerances of test_gpu_logprobs."""
import pytest
import torch

import selective_state_update_gb300 as ssu
from test_gpu_logprobs import DEV, check, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 5, 400])
@pytest.mark.parametrize("value", [-1e10, -1e20, -1e30, 1e12, -1.4e9, 2e8, 3e38, -0.95e38])
def test_constant_rows(libssu, value, rows, dtype):
    """A row that an additive mask covers altogether, and its mirror."""
    x = torch.full((rows, 5000), value, dtype=dtype, device=DEV)
    check(x, torch.arange(rows, device=DEV), 20)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_constant_rows_of_every_size(libssu, sign):
    x = sign * torch.exp2(torch.linspace(18.0, 127.9, 800, device=DEV))[:, None].repeat(1, 1003)
    check(x, torch.full((800,), 1002, device=DEV), 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 5, 400])
@pytest.mark.parametrize("value", [1e6, 1.3e9, 1e10, 1e12, 1e20, 1e30, 3e38])
def test_one_large_logit(libssu, value, rows, dtype):
    """One far above the others, and two."""
    x, tok = logits(300, rows, 4099, dtype)
    tok[:] = 777
    x[:, 777] = value
    check(x, tok, 20)
    check(x, (tok + 1), 20)
    x[:, 3001] = value
    check(x, tok, 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", [-1e4, -1e9, -2e9, -1e10, -1e30])
@pytest.mark.parametrize("rows", [3, 400])
def test_masked_by_large_negatives(libssu, rows, low, dtype):
    """Most of a row under an additive mask: whole threads see nothing else."""
    x, tok = logits(310, rows, 30011, dtype)
    x[:, 1500:] += low
    x[0, :1500] += low
    tok[:] = 40
    tok[1] = 20000
    check(x, tok, 20)
