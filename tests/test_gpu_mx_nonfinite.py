"""Infinities and NaN in the microscaled products' operands: they reach the results that their element
enters, and every other result is as exact as without them.

The update's bound is `apply_want`'s (test_gpu_mx): B terms summed twice in fp32, 22-bit pieces of the
elements of G and T = XL G.
"""
import numpy as np
import pytest
import torch

import dash_inputs as di
import matrix_inverse_roots_amd as dash
import mx_ref as ref
import test_gpu_mx as mx
from test_gpu_mx import DEV, FMTS, IDS, f64

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

# stacks that take 64-, 128- and 256-wide kernel tiles, bounds found by the products' own workgroups (B <= 128)
# and by a launch before them (in 1, 4 and 16 parts per block), whole tiles and edges
STACKS = [(3, 64), (300, 128), (3, 192), (60, 256), (2, 576), (2, 1024), (20, 1088)]


def update(N, B, fmt, size, seed):
    """Random roots with fp32 diagonals and gradients of magnitude `size`."""
    rng = di.rng(seed)
    s = {"N": N, "B": B, "fmt": fmt}
    few = min(N, 3)  # (blocks repeat: codes are made on the host)
    rep = lambda t: t.repeat(-(-N // few), 1, 1)[:N].contiguous()
    for side in "LR":
        q, b, _ = mx.random_codes(rng, few, B, B, fmt)
        s[side], s[side + "s"] = rep(q), rep(b)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    for side in "LR":
        s[side + "d"] = 50 * torch.randn((N, B), generator=gen, device=DEV)
    s["G"] = size * torch.randn((N, B, B), generator=gen, device=DEV)
    return s


def call(s):
    U = torch.full((s["N"], s["B"], s["B"]), 7.0, device=DEV)
    ws = dash.workspace(dash.DASH_OP_APPLY, s["N"], s["B"], device=DEV)
    ws.fill_(0xFF)
    dash.dash_apply_mx(s["L"], s["Ls"], s["R"], s["Rs"], s["G"], s["N"], s["B"], s["fmt"], U, XL_diag=s["Ld"],
                       XR_diag=s["Rd"], ws=ws)
    return U


def check_block(U, s, b, rows, cols):
    """Block b of U: the given rows and columns hold no finite element, the others are within the bound."""
    B = s["B"]
    v = lambda side: ref.values(mx.host(s[side][b]).numpy(), mx.host(s[side + "s"][b]).numpy(), B, s["fmt"])
    L, R, G = v("L") + np.diag(f64(s["Ld"][b])), v("R") + np.diag(f64(s["Rd"][b])), f64(s["G"][b])
    keep_i = [i for i in range(B) if i not in rows]
    keep_j = [j for j in range(B) if j not in cols]
    got = f64(U[b])
    for i in rows:
        assert not np.isfinite(got[i]).any(), (b, i)
    for j in cols:
        assert not np.isfinite(got[:, j]).any(), (b, j)
    L, R = L[keep_i], R[keep_j]
    want, tol = mx.apply_want(L[None], R[None], G[None])
    err = np.abs(got[np.ix_(keep_i, keep_j)] - want[0])
    assert np.all(err <= tol[0]), (b, np.nanmax(err / tol[0]))


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,B", STACKS)
def test_update_inf_in_a_root_diagonal(N, B, fmt):
    """One row (left) or column (right) of the block is lost; gradients of 1e-9 beside it keep their bits."""
    s = update(N, B, fmt, 1e-9, 200 + B)
    b = N // 2
    s["Ld"][b, 5] = INF
    s["Rd"][b, B - 3] = -INF
    U = call(s)
    check_block(U, s, b, [5], [B - 3])
    check_block(U, s, 0 if b else N - 1, [], []) if N > 1 else None


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,B", STACKS)
def test_update_row_that_overflows(N, B, fmt):
    """A row of XL G beyond fp32 leaves the block's others, of 1e5 and more, as they are."""
    s = update(N, B, fmt, 1e5, 210 + B)
    b = N - 1
    s["G"][b, 9] = 1e6
    s["Ld"][b, 9] = 3e38
    U = call(s)
    check_block(U, s, b, [9], [])


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("N,B", STACKS)
def test_update_nonfinite_gradient(N, B, value):
    """A non-finite element of G enters every row of U through its column of T: the block is lost, no other."""
    s = update(N, B, dash.DASH_MX_E4M3, 1e-9, 220 + B)
    b = N // 2
    s["G"][b, 2, 7] = value
    U = call(s)
    assert not bool(torch.isfinite(U[b]).any())
    check_block(U, s, 0 if b else N - 1, [], []) if N > 1 else None


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,B", STACKS)
def test_update_nan_groups_in_roots(N, B, fmt):
    """Scale byte 255 in a row of XL loses that row of U, in a row of XR that column; the byte is no part of
    the block's largest scale."""
    s = update(N, B, fmt, 1e-9, 230 + B)
    b, width = N // 2, 32 if fmt == dash.DASH_MX_E4M3 else 16
    for side, row, group in (("L", 11, B // 32 - 1), ("R", B - 20, 0)):
        s[side + "s"][b, row, group] = 255
        s[side][b, row, width * group:width * (group + 1)] = 0
    U = call(s)
    check_block(U, s, b, [11], [B - 20])


@pytest.mark.parametrize("B", [64, 192, 256])
def test_update_nan_codes_in_roots(B):
    """The E4M3 code that is no number, which the quantiser never writes, reads as NaN."""
    s = update(3, B, dash.DASH_MX_E4M3, 1e-3, 240 + B)
    s["L"][1, 13, 40] = 0x7F
    s["R"][1, 20, 3] = 0xFF
    U = call(s)
    check_block(U, s, 1, [13], [20])
    check_block(U, s, 2, [], [])


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("B", [64, 192, 256])
def test_statistics_nan_groups(B, fmt):
    rng = di.rng(250 + B)
    N, width = 2, 32 if fmt == dash.DASH_MX_E4M3 else 16
    q, s, _ = mx.random_codes(rng, N, B, B, fmt)
    qt, st, _ = mx.random_codes(rng, N, B, B, fmt)
    s[1, 7, 1], st[0, B - 1, 0] = 255, 255
    q[1, 7, width:2 * width] = 0
    qt[0, B - 1, :width] = 0
    if fmt == dash.DASH_MX_E4M3:
        q[0, 3, 5] = 0x7F  # (a code that is no number)
    A = torch.ones((2 * N, B, B), device=DEV)
    dash.dash_update_stats_mx(q, s, qt, st, N, B, fmt, 0.5, A)
    want = torch.zeros_like(A, dtype=torch.bool)
    want[1, 7, :] = want[1, :, 7] = True
    want[N, B - 1, :] = want[N, :, B - 1] = True
    if fmt == dash.DASH_MX_E4M3:
        want[0, 3, :] = want[0, :, 3] = True
    assert torch.equal(torch.isnan(A), want)
    assert bool(torch.isfinite(A[~want]).all())


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("T,out,inp,B", [(70, 96, 96, 128), (2000, 300, 300, 128)])
def test_gradient_nan_groups(T, out, inp, B, fmt):
    """A NaN group of the layer's input loses its 32 columns of the weight, a NaN code its own."""
    rng = di.rng(260 + T)
    width = 32 if fmt == dash.DASH_MX_E4M3 else 16
    q, s, _ = mx.random_codes(rng, 1, T, inp, fmt)
    s[0, T - 1, 1] = 255
    q[0, T - 1, width:2 * width] = 0
    if fmt == dash.DASH_MX_E4M3:
        q[0, 0, 70] = 0xFF
    dY = torch.from_numpy(rng.standard_normal((T, out)).astype(np.float32)).to(DEV)
    G = f64(mx.grad(dY, q, s, fmt, T, out, inp, B)).reshape(-1, B, B)
    bad = np.zeros((out, inp))
    bad[:, 32:64] = 1
    if fmt == dash.DASH_MX_E4M3:
        bad[:, 70] = 1
    assert np.array_equal(np.isnan(G), ref.tiles(bad, B) != 0)


@pytest.mark.parametrize("fmt,step", zip(FMTS, (3.5 * 2.0**126, 248 * 2.0**120)), ids=IDS)
def test_magnitudes_that_round_beyond_fp32(fmt, step):
    """From half a step below 2^128 up an element's value is 2^128: the definition's code, and Inf as a value."""
    big = np.array([step, np.nextafter(np.float32(step), np.float32(0)), torch.finfo(torch.float32).max,
                    torch.finfo(torch.bfloat16).min, -1.0], np.float32)
    x = np.zeros((5, 40), np.float32)
    x[:, 3] = big
    x[:, 35] = 2.0  # (another group)
    c, s = dash.mx_buffers(1, 5, 40, fmt, device=DEV)
    dash.dash_mx_quantize(torch.from_numpy(x).to(DEV), 1, 5, 40, fmt, c, s)
    code, byte = ref.quantize(x[None], fmt)
    assert np.array_equal(mx.host(c).numpy(), ref.pack(code, fmt)) and np.array_equal(mx.host(s).numpy(), byte)
    want = ref.values(ref.pack(code, fmt), byte, 40, fmt)[0]
    assert want[0, 3] == 2.0**128 and want[1, 3] < 2.0**128
    for dtype in (torch.float32, torch.bfloat16):
        v = torch.empty((1, 5, 40), dtype=dtype, device=DEV)
        dash.dash_mx_dequantize(c, s, 1, 5, 40, fmt, v)
        with np.errstate(over="ignore"):
            assert np.array_equal(f64(v)[0], want.astype(np.float32).astype(np.float64))
