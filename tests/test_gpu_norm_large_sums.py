"""x + res beyond fp32's range is an Inf of its row, whatever the row's length."""
import pytest
import torch

from gpu_helpers import DEV
from test_gpu_norm import norm, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 7, 8, 263, 4096, 33000])
def test_a_sum_beyond_fp32(n, dtype):
    T = 6
    x, r = randn(1, T, n, dtype=dtype), randn(2, T, n, dtype=dtype)
    clean = norm(x, r)
    at = n // 2
    x[2, at] = r[2, at] = 3e38
    x[4, at] = r[4, at] = -3e38
    h, y, codes, scales, rstd = norm(x, r)
    rest = [0, 1, 3, 5]
    for a, b in zip((h, y, codes[0], scales[0], rstd), (clean[0], clean[1], clean[2][0], clean[3][0], clean[4])):
        assert torch.equal(a[rest], b[rest])
    for row, inf in ((2, float("inf")), (4, -float("inf"))):
        others = [j for j in range(n) if j != at]
        assert float(h[row, at]) == inf and float(rstd[row]) == 0.0
        assert bool(y[row, at].isnan()) and not bool(y[row, others].any())
        assert int((scales[0, row] == 255).sum()) == 1 and int(scales[0, row, at // 32]) == 255
        assert not bool((codes[0, row] & 0x7f).any())
