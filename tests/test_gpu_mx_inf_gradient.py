"""Infinities in dY give the infinities and NaN of their sums, and its largest finite magnitudes their
products, or Inf where those are beyond fp32."""
import numpy as np
import pytest
import torch

import dash_inputs as di
import matrix_inverse_roots_amd as dash
import mx_ref as ref
import test_gpu_mx as mx
from test_gpu_mx import DEV, FMTS, IDS, TYPES, U, f64

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
    # finite, in rows of their own: their products reach beyond fp32, and the parts of one may differ in sign
    large = {61: torch.finfo(dtype).max}
    if dtype == torch.float32:
        large.update({60: 3.4e38, 62: 2.0**126 * (1 + 0.75 * 2.0**-7)})
    for i, x in large.items():
        dY[6, i] = x
    G = f64(mx.grad(dY, q, s, fmt, T, out, inp, B)).reshape(-1, B, B)
    # the infinite elements' terms alone decide the rows that hold one
    d = f64(dY)
    want = np.zeros((out, inp))
    with np.errstate(invalid="ignore"):
        for t, i in np.argwhere(np.isinf(d)):
            want[i] += d[t, i] * X[0][t]
    rows = lambda keep: ref.tiles(np.repeat(np.isin(np.arange(out), keep)[:, None], inp, 1).astype(float), B) != 0
    held, lone = rows(np.flatnonzero(np.isinf(d).any(0))), rows(list(large))
    want = ref.tiles(want, B)
    assert np.array_equal(np.isnan(G[held]), np.isnan(want[held]))
    inf = held & np.isinf(want)
    assert np.array_equal(G[inf], want[inf])
    assert np.all(np.isfinite(G[~held & ~lone]))
    # a large finite element: its product where fp32 holds it, else Inf of its sign
    big = np.zeros((out, inp))
    for i in large:
        big[i] = d[6, i] * X[0][6]
    big = ref.tiles(big, B)
    assert np.all(np.isfinite(G[lone & (np.abs(big) < 3.3e38)]))
    over = lone & (np.abs(big) > 3.5e38)
    assert np.array_equal(G[over], np.sign(big[over]) * np.inf)
    # and to fp32's sums of 3 T parts, joined in up to 260 (the row's other terms are below 2^-17 of these)
    clear = lone & (np.abs(big) < 3.3e38) & (np.abs(big) > 1e6 * T * np.abs(X[0]).max())
    assert np.all(np.abs(G[clear] - big[clear]) <= ((3 * T + 260) * U + 2.0**-17) * np.abs(big[clear]))
