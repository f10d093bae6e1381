"""The norm of rows whose squares leave fp32's range, held to test_gpu_norm's tolerances."""
import pytest
import torch

from test_gpu_norm import check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant", ["none", "row", "block"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hidden", [8, 1000, 2565, 4096, 8192, 20001])
def test_large_values(libssu, hidden, dtype, quant):
    """Between ordinary rows; one large value among ordinary ones too."""
    x, w, res = problem(600 + hidden, 12, hidden, dtype)
    for row, size in enumerate((1e15, 1e17, 3e18, 1e20, 1e25, 1e30, 1e36)):
        x[row] *= size / float(x[row].float().abs().max())
        res[row] *= size / float(res[row].float().abs().max())
    x[8, hidden // 2] = 1e22
    res[9, 0] = -1e37
    check(x, w, res, quant)
    check(x, w, None, quant)
