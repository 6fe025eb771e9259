"""The update on gradients whose rows and columns differ by many powers of two inside a block.

G and T = XL G go into the products as two binary16 pieces under one power of two per block.  With 2^e x
in binary16's range, 2^13 <= 2^e max|x| < 2^14, the pieces' sum differs from 2^e x by the second rounding
alone: 2^-11 of a remainder that is at most 2^-11 |2^e x|, or 2^-25 (half of binary16's smallest number) where
the remainder is subnormal.  So x enters with an error of at most 2^-22 |x| + 2^-38 max|x|, and

  |U^ - U| <= 2 (B + 4) 2^-23 |XL| |G| |XR|^T                      (fp32 sums and 22 bits, as in test_gpu_mx)
              + 2^-38 max|G| |XL| 1 |XR|^T + 2^-38 max|T| 1 |XR|^T   (the block's own resolution).
"""
import numpy as np
import pytest
import torch

import dash_inputs as di
import matrix_inverse_roots_amd as dash
import test_gpu_mx as mx
from test_gpu_mx import DEV, FMTS, IDS, U, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,B", [(2, 64), (300, 128), (2, 192), (60, 256), (1, 1024)])
def test_rows_and_columns_of_many_magnitudes(N, B, fmt):
    rng = di.rng(330 + B)
    ql, sl, L = mx.random_codes(rng, 1, B, B, fmt)
    qr, sr, R = mx.random_codes(rng, 1, B, B, fmt)
    dl, dr = (rng.standard_normal((1, B)).astype(np.float32) * 50 for _ in range(2))
    L, R = L + dl[:, :, None] * np.eye(B), R + dr[:, :, None] * np.eye(B)
    G = rng.standard_normal((1, B, B))
    G *= np.exp2(-10.0 * (np.arange(B) % 5))[None, None, :]  # columns at 1 .. 2^-40 of the block
    G *= np.exp2(-15.0 * (np.arange(B) % 3))[None, :, None]  # and rows at 1 .. 2^-30
    G = G.astype(np.float32)
    rep = lambda t: t.expand(N, *t.shape[1:]).contiguous()
    Gd = rep(torch.from_numpy(G).to(DEV))
    dl, dr = (rep(torch.from_numpy(d).to(DEV)) for d in (dl, dr))
    got = torch.full((N, B, B), float("nan"), device=DEV)
    ws = dash.workspace(dash.DASH_OP_APPLY, N, B, device=DEV)
    ws.fill_(0xFF)
    dash.dash_apply_mx(rep(ql), rep(sl), rep(qr), rep(sr), Gd, N, B, fmt, got, XL_diag=dl, XR_diag=dr, ws=ws)
    g = G[0].astype(np.float64)
    T = L[0] @ g
    want = T @ R[0].T
    one = np.ones((B, B))
    tol = 2 * (B + 4) * U * (np.abs(L[0]) @ np.abs(g) @ np.abs(R[0]).T)
    tol += 2.0**-38 * (np.abs(g).max() * (np.abs(L[0]) @ one) + np.abs(T).max()) @ np.abs(R[0]).T
    for i in {0, N // 2, N - 1}:
        err = np.abs(f64(got[i]) - want)
        assert np.all(err <= tol), (i, np.max(err / tol))


@pytest.mark.parametrize("fmt,top", zip(FMTS, (6.0, 448.0)), ids=IDS)
@pytest.mark.parametrize("N,B", [(2, 64), (2, 192), (60, 256)])
def test_roots_of_many_scales(N, B, fmt, top):
    """Root groups from 2^-60 of the block's largest scale up: an element is off by half of binary16's smallest
    number where the largest scale's elements are 2^13 and more, 2^-38 of what that scale can hold."""
    rng = di.rng(340 + B)
    ql, sl, L = mx.random_codes(rng, 1, B, B, fmt, 75, 136)
    qr, sr, R = mx.random_codes(rng, 1, B, B, fmt, 75, 136)
    G = rng.standard_normal((1, B, B)).astype(np.float32)
    rep = lambda t: t.expand(N, *t.shape[1:]).contiguous()
    got = torch.full((N, B, B), float("nan"), device=DEV)
    ws = dash.workspace(dash.DASH_OP_APPLY, N, B, device=DEV)
    dash.dash_apply_mx(rep(ql), rep(sl), rep(qr), rep(sr), rep(torch.from_numpy(G).to(DEV)), N, B, fmt, got, ws=ws)
    g, l, r = np.abs(G[0].astype(np.float64)), np.abs(L[0]), np.abs(R[0])
    low = [2.0**-38 * top * 2.0 ** (int(s.max()) - 127) for s in (sl, sr)]
    T = np.abs(L[0] @ G[0].astype(np.float64))
    one = np.ones((B, B))
    want = L[0] @ G[0].astype(np.float64) @ R[0].T
    tol = 2 * (B + 4) * U * (l @ g @ r.T)
    tol += 2.0**-38 * (g.max() * (l @ one) + T.max()) @ r.T
    tol += low[0] * (one @ g) @ r.T + (l @ g) @ (low[1] * one)
    err = np.abs(f64(got[N - 1]) - want)
    assert np.all(err <= tol), np.max(err / tol)
