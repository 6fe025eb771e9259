"""Infinities in dY, and magnitudes that its bfloat16 pieces cannot hold, give the infinities and NaN of the
same sum in 64 bits."""
import numpy as np
import pytest
import torch

import dash_inputs as di
import matrix_inverse_roots_amd as dash
import mx_ref as ref
import test_gpu_mx as mx
from test_gpu_mx import DEV, FMTS, IDS, TYPES, f64

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,out,inp,B", [(70, 96, 96, 128), (3000, 300, 200, 128), (90, 2050, 7000, 512)])
def test_inf_in_dy(T, out, inp, B, dtype, fmt):
    """An Inf times a positive element is Inf, times a negative one -Inf, times zero NaN; so is the sum."""
    rng = di.rng(270 + T)
    q, s, X = mx.random_codes(rng, 1, T, inp, fmt)
    dY = torch.from_numpy(rng.standard_normal((T, out))).to(DEV).to(dtype)
    dY[20, 9] = INF
    dY[T - 1, out - 1] = -INF
    dY[3, 40], dY[4, 40] = INF, INF  # sums of two infinities: NaN where they differ in sign
    if dtype == torch.float32:
        dY[5, 60] = 3.4e38  # above every bfloat16: counts as Inf
    dY[6, 61] = torch.finfo(dtype).max if dtype != torch.float32 else 3.38e38  # the largest that does not
    G = f64(mx.grad(dY, q, s, fmt, T, out, inp, B)).reshape(-1, B, B)
    # by rules: terms of the infinite elements alone decide the rows that hold one
    d = f64(dY)
    d[np.abs(d) > 3.39e38] *= INF
    want = np.zeros((out, inp))
    with np.errstate(invalid="ignore"):
        for t, i in np.argwhere(np.isinf(d)):
            want[i] += d[t, i] * X[0][t]
    want = ref.tiles(want, B)
    row = np.zeros((out, inp))
    row[np.isinf(d).any(0)] = 1
    row = ref.tiles(row, B) != 0
    assert np.array_equal(np.isnan(G[row]), np.isnan(want[row]))
    inf = row & np.isinf(want)
    assert np.array_equal(G[inf], want[inf])
    one = np.zeros((out, inp))
    one[61] = 1
    one = ref.tiles(one, B) != 0
    big = ref.tiles(np.outer(np.eye(out)[61], d[6, 61] * X[0][6]), B)
    over = one & (np.abs(big) > 3.5e38)
    assert np.all(np.isfinite(G[~row & ~one]))
    assert np.all(np.isfinite(G[one & (np.abs(big) < 3e38)])) and np.all(np.isinf(G[over]))
