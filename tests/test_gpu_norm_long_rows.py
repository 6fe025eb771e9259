"""The gradient of rows of millions of elements, whose sums must not lose bits with the row's length.

Tolerance, u = 2^-24, apart from the row's length: xhat and m carry u each; the mean adds at most 8 products in 32 bits
(10 u with theirs) and 64 bits from there, and is rounded and scaled in 32 (3 u): 13 u of the mean magnitude.  Then
as for shorter rows: 4u (|m| + |xhat c|) rstd, u |dx| and half a step of the type."""
import pytest
import torch

from gpu_helpers import DEV
from test_gpu_norm import LEAST, NAMES, TYPES, U, back, half, randn

pytestmark = pytest.mark.gpu


def check(dy, h, rstd, gain, dh, dx):
    r = rstd.double()[:, None]
    xhat, m = h.double() * r, dy.double() * (1 if gain is None else gain.double())
    c = (m * xhat).mean(1, keepdim=True)
    want = r * (m - xhat * c) + (0 if dh is None else dh.double())
    tol = 4 * U * r * (m.abs() + (xhat * c).abs()) + r * xhat.abs() * 13 * U * (m * xhat).abs().mean(1, keepdim=True)
    tol = tol + (U + half(dy.dtype)) * (want.abs() + tol) + LEAST[dy.dtype]
    assert bool(((dx.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n", [40001, (1 << 20) + 3, (1 << 23) + 5])
def test_mean_of_a_long_row(n, dtype):
    """Products of one size, whose sum rounds the same way in every step, and random ones."""
    for k in range(2):
        h = torch.full((2, n), 1.3, dtype=dtype, device=DEV) if k == 0 else randn(1, 2, n, dtype=dtype)
        dy = torch.full((2, n), 0.7, dtype=dtype, device=DEV) if k == 0 else randn(2, 2, n, dtype=dtype)
        rstd = torch.tensor([0.77, 1.01], device=DEV)
        gain = None if k == 0 else 1 + randn(3, n, scale=0.3)
        dgain = torch.empty(n, device=DEV)
        dx = back(dy, h, rstd, gain, dgain=dgain)
        check(dy, h, rstd, gain, None, dx)
        terms = dy.double() * h.double() * rstd.double()[:, None]
        assert bool(((dgain.double() - terms.sum(0)).abs() <= 8 * U * terms.abs().sum(0)).all())
        dh = randn(4, 2, n, dtype=dtype)
        check(dy, h, rstd, gain, dh, back(dy, h, rstd, gain, dh))
