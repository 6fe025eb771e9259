"""The norm with the residual's addition and a microscaled output, and its gradient, against 64-bit
arithmetic.

Tolerances, u = 2^-24 (half a step of fp32).  h = x + res is off by u |h| before its own rounding.  The sum
of squares adds terms of one sign: 2u from h, at most 8 roundings in a piece of 8, 64 bits between pieces;
its root halves that, rstd's own rounding adds u: 6u.  y = (h rstd) gain adds u for h and 2u for the products:
9u, 10u with the second order.  A stored value adds half a step of its type, relative (eps / 2), or half of its
least magnitude.

The gradient.  xhat and m carry u each.  The mean c adds n products in chains of at most 32 in a thread (n / 1024
+ 8 for rows longer than 16384), 6 steps in a wave and up to 16 waves: L = chain + 24 roundings of the sum of
magnitudes.  dx = dh + rstd (m - xhat c): 4u (|m| + |xhat c|) rstd + rstd |xhat| (L u mean |m xhat|) + u |dx|,
then its own rounding.  dgain adds rows in at least min(T, 256) and at most 512 shares, in each rows side by side
(the wider the rows the fewer) whose chains take every `side by side`-th row: at most T / 256 + 1 of them, which the
joins of those (9 halvings) and of the shares (64 bits) follow; few rows in chains of T / 32: (T / 256 + 260) u of
the sum of magnitudes covers all."""
import numpy as np
import pytest
import torch

import matrix_inverse_roots_amd as dash
import mx_ref as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

U = 2.0**-24
EPS = 1e-5
TYPES = [torch.float32, torch.bfloat16, torch.float16]
FMTS = [dash.DASH_MX_E4M3, dash.DASH_MX_E2M1]
IDS = ["e4m3", "e2m1"]
LEAST = {torch.float32: 2.0**-149, torch.bfloat16: 2.0**-133, torch.float16: 2.0**-24}
NAMES = {torch.float32: "fp32", torch.bfloat16: "bf16", torch.float16: "fp16"}
# (T, n): one row, one element; around a piece, a group, a wave; rows in every number of threads; long ones
SIZES = [(1, 1), (3, 2), (300, 7), (5, 8), (64, 9), (2, 31), (33, 32), (7, 33), (3, 63), (600, 64), (1, 255),
         (513, 263), (9, 512), (700, 1001), (1, 2048), (520, 2047), (4, 4104), (515, 4096), (3, 8192), (2, 8195),
         (2, 16385), (513, 12000), (2, 32768), (1, 33000), (2, 65537)]


def half(dtype):
    return torch.finfo(dtype).eps / 2


def randn(seed, *shape, scale=1.0, dtype=torch.float32):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(shape, generator=gen, device=DEV)).to(dtype)


def pitched(t, pad):
    """t's values as the columns of a wider buffer (of 77s)."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 77, dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def definition(x, res, gain, eps=EPS):
    h = x.double() + (0 if res is None else res.double())
    rstd = ((h * h).mean(1) + eps) ** -0.5
    return h, rstd, h * rstd[:, None] * (1 if gain is None else gain.double())


def norm(x, res=None, gain=None, fmt=FMTS[0], eps=EPS, y=True, in_place=None):
    """The call's (h, y, codes, scales, rstd)."""
    T, n = x.shape
    h = in_place if in_place is not None else torch.empty_like(x)
    y = torch.empty_like(x) if y else None
    codes, scales = dash.mx_buffers(1, T, n, fmt, device=DEV)
    rstd = torch.empty(T, device=DEV)
    dash.dash_rmsnorm(x, T, n, eps, res=res, gain=gain, h=h, y=y, fmt=fmt, codes=codes, scales=scales, rstd=rstd)
    torch.cuda.synchronize()
    return h, y, codes, scales, rstd


def check_codes(codes, scales, want, fmt, off=10 * U):
    """The microscaled rows stand for `want`, known up to `off` relative, as the format defines."""
    want = want.cpu().numpy()
    T, n = want.shape
    g = -(-n // 32)
    pad = np.zeros((T, g * 32))
    pad[:, :n] = want
    top = np.abs(pad).reshape(T, g, 32).max(-1)

    def byte(t):
        _, b = ref.quantize(np.repeat(t[..., None], 32, -1).reshape(T, g * 32), fmt)
        return b

    scales = scales.cpu().numpy()[0].astype(np.int64)
    assert np.all(scales >= byte(top * (1 - off))) and np.all(scales <= byte(top * (1 + off)))
    got = ref.values(codes.cpu().numpy()[0], scales, g * 32, fmt)
    assert not got[:, n:].any()
    step = np.repeat(2.0 ** (scales - 127.0), 32, -1)  # the scale
    least = 2.0**-10 if fmt == dash.DASH_MX_E4M3 else 0.25  # half of the least element
    rel = 2.0**-4 if fmt == dash.DASH_MX_E4M3 else 0.25
    tol = off * np.abs(pad) + np.maximum(rel * (1 + off) * np.abs(pad), least * step)
    assert np.all(np.abs(got - pad) <= tol)


def check_norm(x, res, gain, out, fmt, eps=EPS):
    h, y, codes, scales, rstd = out
    wh, wr, wy = definition(x, res, gain, eps)
    e, least = half(x.dtype), LEAST[x.dtype]
    assert bool(((h.double() - wh).abs() <= (U + e) * wh.abs() + least).all())
    assert bool(((rstd.double() - wr).abs() <= 6 * U * wr).all())
    if y is not None:
        assert bool(((y.double() - wy).abs() <= (10 * U + e) * wy.abs() + least).all())
    check_codes(codes, scales, wy, fmt)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("T,n", SIZES)
def test_norm(T, n, dtype):
    seed = 1000 + n
    for i, (res, gain_type, pad, fmt) in enumerate(((True, dtype, 0, FMTS[0]), (False, None, 3, FMTS[1]),
                                                    (True, torch.float32, 8, FMTS[1]),
                                                    (True, torch.bfloat16, 1, FMTS[0]))):
        x = pitched(randn(seed + i, T, n, scale=3, dtype=dtype), pad)
        r = pitched(randn(seed + 10 + i, T, n, dtype=dtype), 2 * pad) if res else None
        gain = None if gain_type is None else (1 + randn(seed + 20, n, scale=0.3)).to(gain_type)
        check_norm(x, r, gain, norm(x, r, gain, fmt), fmt)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("T,n", [(3, 5), (70, 263), (600, 2048), (2, 33001)])
def test_h_in_the_place_of_an_input(T, n, dtype):
    x, r = randn(30, T, n, dtype=dtype), randn(31, T, n, dtype=dtype)
    gain = 1 + randn(32, n, scale=0.3)
    want = norm(x, r, gain)
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        got = norm(a, b, gain, in_place=(a, b)[which])
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal((b, a)[which], (r, x)[which])


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("T,n", [(5, 6), (9, 263), (300, 1024), (2, 40000)])
def test_codes_are_those_of_64_bits(T, n, dtype, fmt):
    """Every byte is the definition's: y is rounded once.  (The call's y is within 2^-44 of it, at fewer than 2^19
    elements of which one in 2^20 a step of 2^-24 lies next to a border: 2^-20 of them on the other side.)"""
    for res in (False, True):
        x, gain = randn(40, T, n, scale=5, dtype=dtype), 1 + randn(41, n, scale=0.3)
        r = randn(42, T, n, dtype=dtype) if res else None
        _, _, codes, scales, _ = norm(x, r, gain, fmt)
        want, byte = ref.quantize(definition(x, r, gain)[2].cpu().numpy(), fmt)
        assert np.array_equal(codes.cpu().numpy()[0], ref.pack(want, fmt))
        assert np.array_equal(scales.cpu().numpy()[0], byte)


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n", [7, 64, 1024, 8208, 33024])
def test_codes_next_to_borders(n, dtype, fmt):
    """Rows of one magnitude (of any size), for which y = +-gain, and gains one step of 2^-24 to either side of the
    borders between codes (and of scales, in groups of their own)."""
    t = ref.grid(fmt)
    mid = (t[1:] + t[:-1]) / 2
    rng = np.random.default_rng(7)
    g = rng.choice(mid[len(mid) // 3:], n) / 4
    g[32::64] = ref.TOP[fmt] / 8  # (the groups' largest elements: some are borders of scales)
    gain = np.nextafter(g.astype(np.float32), (2 * rng.integers(0, 2, n) * g.max()).astype(np.float32))
    assert gain.dtype == np.float32 and np.all(gain != g)
    T = 40
    size = torch.tensor(rng.uniform(0.1, 100, T), device=DEV)[:, None].to(dtype)
    sign = torch.tensor(rng.choice([-1.0, 1.0], (T, n)), device=DEV).to(dtype)
    x = size * sign
    for res in (None, (size * 0.377).to(dtype) * sign):
        got = norm(x, res, torch.tensor(gain, device=DEV), fmt, eps=0.0, y=False)
        want, byte = ref.quantize(sign.double().cpu().numpy() * gain.astype(np.float64), fmt)
        assert np.array_equal(got[2].cpu().numpy()[0], ref.pack(want, fmt)), res is None
        assert np.array_equal(got[3].cpu().numpy()[0], byte)


def test_each_output_alone():
    T, n = 40, 300
    x, r, gain = (randn(50 + i, *s, dtype=torch.bfloat16) for i, s in enumerate(((T, n), (T, n), (n,))))
    h, y, codes, scales, rstd = norm(x, r, gain)
    got = [torch.empty_like(v) for v in (h, y, codes, scales, rstd)]
    dash.dash_rmsnorm(x, T, n, EPS, res=r, gain=gain, h=got[0])
    dash.dash_rmsnorm(x, T, n, EPS, res=r, gain=gain, y=got[1])
    dash.dash_rmsnorm(x, T, n, EPS, res=r, gain=gain, codes=got[2], scales=got[3])
    dash.dash_rmsnorm(x, T, n, EPS, res=r, gain=gain, rstd=got[4])
    assert all(torch.equal(a, b) for a, b in zip(got, (h, y, codes, scales, rstd)))


@pytest.mark.parametrize("n", [4, 40, 263, 4096, 33000])
def test_large_and_small_rows(n):
    """Rows whose squares leave fp32's range on either side, rows of one large element, rows of zeros."""
    x = randn(60, 8, n)
    for r, s in enumerate((1e30, 1e38, 1e-25, 1e-38, 1.0)):
        x[r] = (x[r].double() * s).clamp(-3e38, 3e38).float()
    x[5] = 0
    x[6] = 0
    x[6, n // 2] = 1e25
    out = norm(x, eps=0.0 if n == 40 else 1e-12)
    keep = [0, 1, 2, 3, 4, 6, 7] if n == 40 else list(range(8))
    wh, wr, wy = definition(x, None, None, 0.0 if n == 40 else 1e-12)
    assert torch.equal(out[0], x)
    # (rstd may lie below 2^-126, where a step is 2^-149)
    tol = 6 * U * wr + 2.0**-150
    assert bool(((out[4].double() - wr).abs() <= tol)[keep].all())
    y_tol = 10 * U * wy.abs() + 2.0**-150 * (1 + wh.abs())
    assert bool(((out[1].double() - wy).abs() <= y_tol)[keep].all())
    if n == 40:  # eps = 0 and zeros: 0 / 0
        assert bool(torch.isinf(out[4][5])) and bool(torch.isnan(out[1][5]).all())
        assert bool((out[3][0, 5] == 255).all()) and not bool(out[2][0, 5].any())


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("n", [6, 64, 1001, 33000])
def test_rows_that_are_not_finite(n, dtype):
    """A NaN or an Inf stays in its row; the others keep their bits."""
    T = 12
    x, gain = randn(70, T, n, dtype=dtype), 1 + randn(71, n, scale=0.3)
    clean = norm(x, None, gain)
    bad = x.clone()
    bad[2, n - 1] = float("nan")
    bad[5, n // 2] = float("inf")
    bad[6, 0] = -float("inf")
    h, y, codes, scales, rstd = norm(bad, None, gain)
    rest = [i for i in range(T) if i not in (2, 5, 6)]
    for a, b in zip((h, y, codes[0], scales[0], rstd), (clean[0], clean[1], clean[2][0], clean[3][0], clean[4])):
        assert torch.equal(a[rest], b[rest])
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(rstd[2])) and bool((scales[0, 2] == 255).all())
    for r, at in ((5, n // 2), (6, 0)):
        assert float(rstd[r]) == 0.0 and bool(torch.isnan(y[r, at]))
        others = [j for j in range(n) if j != at]
        assert not bool(y[r, others].any())
        assert int((scales[0, r] == 255).sum()) == 1 and int(scales[0, r, at // 32]) == 255
        assert not bool((codes[0, r] & 0x7f).any())


def test_norm_past_32_bit_offsets():
    """Rows beyond 2^32 elements of a wide buffer."""
    T, n, ld = 70001, 40, 65536
    wide = torch.zeros((T, ld), dtype=torch.bfloat16, device=DEV)
    x = wide[:, :n]
    x.copy_(randn(80, T, n, dtype=torch.bfloat16))
    got = norm(x)
    want = norm(x.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    dy = randn(81, T, n, dtype=torch.bfloat16)
    dx, dgain = torch.empty_like(dy), torch.empty(n, device=DEV)
    ws = dash.rmsnorm_backward_workspace(T, n, device=DEV)
    dash.dash_rmsnorm_backward(dy, x.contiguous(), got[4], T, n, dx, dgain=dgain, ws=ws)
    dash.dash_rmsnorm_backward(dy, x, got[4], T, n, x_out := wide[:, 100:100 + n], ws=ws)
    assert torch.equal(x_out, dx) and not bool(wide[:, 100 + n:].any()) and not bool(wide[:, n:100].any())


LARGE = [(30001, 2047, torch.bfloat16), (9000, 8192, torch.bfloat16), (2300, 32000, torch.float16),
         (30000, 2048, torch.float32), (15001, 4095, torch.float32), (7000, 8192, torch.float32),
         (4000, 16384, torch.float32)]
LARGE_IDS = ["%dx%d-%s" % (T, n, NAMES[t]) for T, n, t in LARGE]


@pytest.mark.parametrize("T,n,dtype", LARGE, ids=LARGE_IDS)
def test_large_calls_equal_their_parts(T, n, dtype):
    """A row's results do not depend on how many others there are (calls beyond the caches' size store past them)."""
    x, r = randn(130, T, n, dtype=dtype), randn(131, T, n, dtype=dtype)
    gain = 1 + randn(132, n, scale=0.3)
    whole = norm(x, r, gain)
    for a, b in ((0, 700), (T // 2, T // 2 + 601), (T - 650, T)):
        part = norm(x[a:b], r[a:b], gain)
        for w, p in zip(whole, part):
            w = w[0] if w.dim() == 3 else w
            assert torch.equal(w[a:b], p[0] if p.dim() == 3 else p)


# ------------------------------------------------------------------------------------------------
# The gradient
# ------------------------------------------------------------------------------------------------


def check_back(dy, h, rstd, gain, dh, dx, dgain, old=None):
    T, n = dy.shape
    d, r = dy.double(), rstd.double()[:, None]
    xhat = h.double() * r
    m = d * (1 if gain is None else gain.double())
    c = (m * xhat).mean(1, keepdim=True)
    want = r * (m - xhat * c) + (0 if dh is None else dh.double())
    L = max(32, n / 1024 + 8) + 24
    tol = 4 * U * r * (m.abs() + (xhat * c).abs()) + r * xhat.abs() * L * U * (m * xhat).abs().mean(1, keepdim=True)
    tol = tol + (U + half(dy.dtype)) * (want.abs() + tol) + LEAST[dy.dtype]
    assert bool(((dx.double() - want).abs() <= tol).all())
    if dgain is not None:
        want = (d * xhat).sum(0) + (0 if old is None else old.double())
        tol = (T / 256 + 260) * U * (d * xhat).abs().sum(0) + U * want.abs() + 2.0**-149
        assert bool(((dgain.double() - want).abs() <= tol).all())


def back(dy, h, rstd, gain=None, dh=None, dx=None, dgain=None, accumulate=False):
    T, n = dy.shape
    dx = torch.empty_like(dy) if dx is None else dx
    ws = dash.rmsnorm_backward_workspace(T, n, device=DEV)
    dash.dash_rmsnorm_backward(dy, h, rstd, T, n, dx, gain=gain, dh=dh, dgain=dgain, accumulate=accumulate, ws=ws)
    torch.cuda.synchronize()
    return dx


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("T,n", SIZES + [(5000, 40), (20000, 3), (1500, 520)])
def test_gradient(T, n, dtype):
    seed = 2000 + n
    for i, (with_dh, gain_type, pad, accumulate) in enumerate(((True, dtype, 0, False), (False, None, 3, True),
                                                               (True, torch.float32, 8, True),
                                                               (False, torch.float16, 1, False))):
        h = pitched(randn(seed + i, T, n, scale=3, dtype=dtype), pad)
        rstd = ((h.double() ** 2).mean(1) + EPS).rsqrt().float()
        dy = pitched(randn(seed + 10 + i, T, n, scale=0.1, dtype=dtype), pad)
        dh = pitched(randn(seed + 20 + i, T, n, scale=0.1, dtype=dtype), 2 * pad) if with_dh else None
        gain = None if gain_type is None else (1 + randn(seed + 30, n, scale=0.3)).to(gain_type)
        old = randn(seed + 40, n)
        dgain = old.clone()
        dx = back(dy, h, rstd, gain, dh, dgain=dgain, accumulate=accumulate)
        check_back(dy, h, rstd, gain, dh, dx, dgain, old if accumulate else None)
        again = torch.full((n,), 5.0, device=DEV)
        dx2 = back(dy, h, rstd, gain, dh, dgain=again)
        assert torch.equal(dx, dx2)
        if not accumulate:
            assert torch.equal(again, dgain)  # equal calls, equal bits
        assert torch.equal(back(dy, h, rstd, gain, dh), dx)  # without dgain


@pytest.mark.parametrize("T,n,dtype", LARGE, ids=LARGE_IDS)
def test_large_gradients(T, n, dtype):
    h, dy, dh = (randn(140 + i, T, n, dtype=dtype) for i in range(3))
    rstd = torch.cat([((h[i:i + 1000].double() ** 2).mean(1) + EPS).rsqrt().float() for i in range(0, T, 1000)])
    gain, dgain = 1 + randn(143, n, scale=0.3), torch.empty(n, device=DEV)
    dx = back(dy, h, rstd, gain, dh, dgain=dgain)
    want, mag = (torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, T, 1000):
        rows = slice(i, i + 1000)
        check_back(dy[rows], h[rows], rstd[rows], gain, dh[rows], dx[rows], None)
        terms = dy[rows].double() * h[rows].double() * rstd[rows].double()[:, None]
        want += terms.sum(0)
        mag += terms.abs().sum(0)
    assert bool(((dgain.double() - want).abs() <= (T / 256 + 260) * U * mag).all())
    part = back(dy[:600], h[:600], rstd[:600], gain, dh[:600])
    assert torch.equal(part, dx[:600])


@pytest.mark.parametrize("T,n", [(1, 8), (100, 1001), (512, 2048), (512, 5001), (300, 16000), (513, 2048)])
def test_gradient_of_few_rows(T, n):
    """dgain of few rows by one launch, or (dx in dy's place) by two: near each other and the definition."""
    for dtype in TYPES:
        h, dy = randn(150, T, n, dtype=dtype), randn(151, T, n, dtype=dtype)
        rstd = ((h.double() ** 2).mean(1) + EPS).rsqrt().float()
        old = randn(152, n)
        for accumulate in (False, True):
            one, two, over = old.clone(), old.clone(), dy.clone()
            dx = back(dy, h, rstd, dgain=one, accumulate=accumulate)
            assert torch.equal(back(over, h, rstd, dx=over, dgain=two, accumulate=accumulate), dx)
            for dgain in (one, two):
                check_back(dy, h, rstd, None, None, dx, dgain, old if accumulate else None)


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES.get)
@pytest.mark.parametrize("T,n", [(3, 5), (600, 263), (600, 2048), (1, 40001)])
def test_dx_in_the_place_of_an_input(T, n, dtype):
    h, dy, dh = (randn(90 + i, T, n, dtype=dtype) for i in range(3))
    rstd = ((h.double() ** 2).mean(1) + EPS).rsqrt().float()
    want = back(dy, h, rstd, None, dh)
    for which in (0, 1):
        a, b = dy.clone(), dh.clone()
        assert torch.equal(back(a, h, rstd, None, b, dx=(a, b)[which]), want)
        assert torch.equal((b, a)[which], (dh, dy)[which])


@pytest.mark.parametrize("T,n", [(7, 5), (300, 130), (2, 33000)])
def test_gradient_is_a_row_s_own(T, n):
    """A NaN in a row of dy, h or dh stays in that row of dx (and in dgain where it enters)."""
    h, dy, dh = (randn(100 + i, T, n) for i in range(3))
    rstd = ((h.double() ** 2).mean(1) + EPS).rsqrt().float()
    want = back(dy, h, rstd, None, dh)
    for k in range(3):
        bad = [t.clone() for t in (dy, h, dh)]
        bad[k][1, n // 2] = float("nan")
        dgain = torch.empty(n, device=DEV)
        dx = back(bad[0], bad[1], rstd, None, bad[2], dgain=dgain)
        rest = [i for i in range(T) if i != 1]
        assert torch.equal(dx[rest], want[rest])
        assert bool(torch.isnan(dx[1]).all()) if k < 2 else int(torch.isnan(dx).sum()) == 1
        assert int(torch.isnan(dgain).sum()) == (1 if k < 2 else 0)


def test_no_rows():
    n = 40
    x = torch.empty((0, n), device=DEV)
    dash.dash_rmsnorm(x, 0, n, EPS, y=torch.empty((0, n), device=DEV))
    dgain = torch.full((n,), 3.0, device=DEV)
    ws = dash.rmsnorm_backward_workspace(0, n, device=DEV)
    dash.dash_rmsnorm_backward(x, x, torch.empty(0, device=DEV), 0, n, x, dgain=dgain, accumulate=True, ws=ws)
    assert bool((dgain == 3).all())
    dash.dash_rmsnorm_backward(x, x, torch.empty(0, device=DEV), 0, n, x, dgain=dgain, ws=ws)
    assert not bool(dgain.any())


def test_gradient_against_differences():
    """f(x, gain) = sum w tanh(y) in 64 bits: central differences in single inputs and gains."""
    T, n = 6, 70
    x, gain, w = randn(110, T, n).double(), 1 + randn(111, n, scale=0.3).double(), randn(112, T, n).double()

    def f(x, gain):
        return (w * torch.tanh(definition(x, None, gain)[2])).sum()

    y = definition(x, None, gain)[2]
    dy = (w * (1 - torch.tanh(y) ** 2)).float()
    rstd = definition(x, None, gain)[1].float()
    dgain = torch.empty(n, device=DEV)
    dx = back(dy, x.float(), rstd, gain.float(), dgain=dgain)
    step = 1e-4
    for t, j in ((0, 0), (5, 69), (2, 33), (3, 64)):
        e = torch.zeros_like(x)
        e[t, j] = step
        d = float((f(x + e, gain) - f(x - e, gain)) / (2 * step))
        # step^2 f''' / 6 with f''' of some 10; the fp32 inputs and sums: 100 u of values of some 4
        assert abs(float(dx[t, j]) - d) <= 1e-5 * (1 + abs(d)), (t, j)
        d = float((f(x, gain + e[t]) - f(x, gain - e[t])) / (2 * step))
        assert abs(float(dgain[j]) - d) <= 1e-5 * (1 + abs(d)), j


@pytest.mark.parametrize("T,n", [(1, 6), (65, 8), (5, 263), (130, 2000), (515, 264), (2, 33001)])
def test_nothing_is_written_past_the_buffers(T, n):
    """Outputs and exactly sized workspaces end where they say; the columns between rows stay."""
    ld = n + 5

    def guarded(size, dtype):
        buf = torch.full((size + 4096,), 77, dtype=dtype, device=DEV)
        return buf, buf[:size]

    for dtype in TYPES:
        g = -(-n // 32)
        bufs = [guarded((T - 1) * ld + n, dtype) for _ in range(3)]
        h, y, dx = (v.as_strided((T, n), (ld, 1)) for _, v in bufs)
        code, scale = guarded(T * g * 32, torch.uint8), guarded(T * g, torch.uint8)
        rstd, dgain = guarded(T, torch.float32), guarded(n, torch.float32)
        ws = guarded(dash.dash_rmsnorm_backward_workspace(T, n), torch.uint8)
        x, r = randn(120, T, n, dtype=dtype), randn(121, T, n, dtype=dtype)
        dash.dash_rmsnorm(x, T, n, EPS, res=r, h=h, y=y, codes=code[1], scales=scale[1], rstd=rstd[1])
        dash.dash_rmsnorm_backward(r, x, rstd[1], T, n, dx, dgain=dgain[1], ws=ws[1])
        torch.cuda.synchronize()
        for buf, v in (*bufs, code, scale, rstd, dgain, ws):
            assert bool((buf[v.numel():] == 77).all())
        for _, v in bufs:
            if T > 1:
                gaps = v[: (T - 1) * ld].view(T - 1, ld)[:, n:]
                assert bool((gaps == 77).all())
        assert bool(torch.isfinite(dx).all())


def test_wrong_tensors_are_refused():
    x, y = torch.zeros((8, 64), device=DEV), torch.zeros((8, 64), device=DEV)
    f = dash.dash_rmsnorm
    for bad in (x.t(), x.double(), x[:, :32], x[:4], x.int()):
        with pytest.raises(ValueError):
            f(bad, 8, 64, EPS, y=y)
        with pytest.raises(ValueError):
            f(x, 8, 64, EPS, y=bad)
        with pytest.raises(ValueError):
            dash.dash_rmsnorm_backward(x, bad, torch.zeros(8, device=DEV), 8, 64, y)
    with pytest.raises(ValueError):
        f(x, 8, 64, EPS, res=x.bfloat16(), y=y)  # one type
    with pytest.raises(ValueError):
        f(x, 8, 64, EPS, y=y, gain=torch.ones(63, device=DEV))
    with pytest.raises(ValueError):
        f(x, 8, 64, EPS, y=y, gain=torch.ones(64, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        f(x, 8, 64, EPS, y=y, rstd=torch.ones(7, device=DEV))
    with pytest.raises(ValueError):
        f(x, 8, 64, EPS, codes=torch.empty(100, dtype=torch.uint8, device=DEV), scales=y)
    with pytest.raises(dash.DashError):
        f(x, 8, 64, EPS, y=x)
    with pytest.raises(dash.DashError):
        dash.dash_rmsnorm_backward(x, y, torch.zeros(8, device=DEV), 8, 64, y)
