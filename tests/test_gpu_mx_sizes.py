"""Microscaled statistics, update and gradient tiles at block sizes up to the largest, 8192, and with
operands whose sums a truncating matrix unit would get wrong, against 64-bit products.

Tolerances.  A statistic's terms are exact products; the matrix unit adds them to an fp32 accumulator at
least 8 at a time.  For terms of one sign the partial sums rise evenly to the total, so K / 8 additions
that each round by half of 2^-23 of the partial sum are off by at most K / 16 2^-24 of the total (K = 4096:
1.5e-5; sums that drop the bits below their largest addend are off by 7e-5), and mixed signs by no more of
the sum of magnitudes; the epilogue's two products and one addition, and 1 - beta in fp32, add 2^-22.  The
elementwise bounds are test_gpu_mx's.
"""
import pytest
import torch

import dash_inputs as di
import matrix_inverse_roots_amd as dash
import mx_ref as ref
import test_gpu_mx as mx
from test_gpu_mx import DEV, FMTS, IDS, U

pytestmark = pytest.mark.gpu


def device_codes(seed, N, rows, cols, fmt, positive=False, lo=120, hi=134):
    """random_codes made on the device: (codes, scales, values in 64 bits)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    e4 = fmt == dash.DASH_MX_E4M3
    c = torch.randint(0, (128 if e4 else 8) * (1 if positive else 2), (N, rows, cols), generator=gen, device=DEV)
    if e4:
        c[c % 128 == 127] = 0
    s = torch.randint(lo, hi, (N, rows, cols // 32), generator=gen, device=DEV)
    half = 128 if e4 else 8
    t = torch.zeros(half, dtype=torch.float64, device=DEV)
    g = torch.from_numpy(ref.grid(fmt)).double().to(DEV)
    t[:len(g)] = g
    v = torch.where(c >= half, -1.0, 1.0).double() * t[c % half]
    v *= torch.exp2(s.double() - 127).repeat_interleave(32, -1)
    q = c.to(torch.uint8)
    if not e4:
        q = q[..., 0::2] | (q[..., 1::2] << 4)
    return q.contiguous(), s.to(torch.uint8), v


@pytest.mark.parametrize("positive", [False, True], ids=["mixed", "positive"])
@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,B", [(3, 64), (2, 128), (2, 448), (2, 1024), (1, 1600), (1, 2048), (1, 4096), (1, 8192)])
def test_statistics(N, B, fmt, positive):
    q, s, v = device_codes(300 + B, N, B, B, fmt, positive)
    qt, st, vt = device_codes(301 + B, N, B, B, fmt, positive)
    gen = torch.Generator(device=DEV).manual_seed(B)
    A = torch.randn((2 * N, B, B), generator=gen, device=DEV)
    A = A + A.transpose(1, 2)
    old = A.clone()
    beta = 0.5  # (exact, as is 1 - beta)
    dash.dash_update_stats_mx(q, s, qt, st, N, B, fmt, beta, A)
    for i in range(2 * N):
        g = (v if i < N else vt)[i % N]
        want = beta * old[i].double() + (1 - beta) * (g @ g.t().contiguous())
        a = g.abs()
        mag = (1 - beta) * (a @ a.t().contiguous())
        own = beta * old[i].double().abs() + mag
        err = (A[i].double() - want).abs()
        assert bool((err <= B * U * mag + 4 * U * own).all()), i
        assert float(err.norm()) <= (B / 16 * 2.0**-24 + 2.0**-22) * float(own.norm()), (i, float(err.norm() / own.norm()))
        assert torch.equal(A[i], A[i].t())


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,B", [(1, 704), (2, 1024), (40, 1024), (30, 1088), (1, 2048), (1, 8192)])
def test_update(N, B, fmt):
    """Every split of the bounds' launch and every tile width, up to the largest block."""
    few = min(N, 2)
    ql, sl, L = device_codes(310 + B, few, B, B, fmt)
    qr, sr, R = device_codes(311 + B, few, B, B, fmt)
    gen = torch.Generator(device=DEV).manual_seed(B)
    d = 50 * torch.randn((2, few, B), generator=gen, device=DEV)
    G = torch.randn((N, B, B), generator=gen, device=DEV)
    rep = lambda t: t.repeat(-(-N // few), *[1] * (t.dim() - 1))[:N].contiguous()
    got = torch.full((N, B, B), float("nan"), device=DEV)
    ws = dash.workspace(dash.DASH_OP_APPLY, N, B, device=DEV)
    ws.fill_(0xFF)
    dash.dash_apply_mx(rep(ql), rep(sl), rep(qr), rep(sr), G, N, B, fmt, got, XL_diag=rep(d[0]), XR_diag=rep(d[1]),
                       ws=ws)
    for i in {0, 1, N // 2, N - 1} & set(range(N)):
        l, r = (x[i % few].clone() for x in (L, R))
        l.diagonal().add_(d[0, i % few].double())
        r.diagonal().add_(d[1, i % few].double())
        rt, g = r.t().contiguous(), G[i].double()
        want = (l @ g) @ rt
        mag = (l.abs() @ g.abs()) @ rt.abs()
        err = (got[i].double() - want).abs()
        assert bool((err <= 2 * (B + 4) * U * mag).all()), i
        assert float(err.norm()) <= 2e-6 * float(want.norm()), i


@pytest.mark.parametrize("dtype", mx.TYPES, ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,out,inp,B", [(300, 100, 70, 8192), (40, 9000, 160, 8192)])
def test_gradient_largest_tiles(T, out, inp, B, dtype):
    fmt = dash.DASH_MX_E2M1 if out > B else dash.DASH_MX_E4M3
    rng = di.rng(320)
    q, s, X = mx.random_codes(rng, 1, T, inp, fmt)
    dY = torch.from_numpy(rng.standard_normal((T, out))).to(DEV).to(dtype)
    G = mx.grad(dY, q, s, fmt, T, out, inp, B).reshape(-1, B, B)
    d = mx.f64(dY)
    want, mag = (torch.from_numpy(w).to(DEV) for w in (d.T @ X[0], abs(d).T @ abs(X[0])))
    for t in range(G.shape[0]):
        rows = min(B, out - t * B)
        part = slice(t * B, t * B + rows)
        err = (G[t, :rows, :inp].double() - want[part]).abs()
        assert bool((err <= (3 * T + 260) * U * mag[part]).all())
        assert not G[t, rows:].any() and not G[t, :, inp:].any()
