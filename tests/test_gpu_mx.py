"""Microscaled quantisation, statistics, update and gradient tiles on the GPU against their definitions
in 64 bits (mx_ref).

Tolerances.  Quantised codes, scales and fp32 values are exact.  A product's terms are exact and its K
terms are summed in fp32: whatever the order, and with a matrix unit that may truncate where fp32
rounds (one unit of 2^-23 per addition instead of half of one), the sum is off by at most
K 2^-23 sum|terms|; `bound` adds 4 2^-23 of the result's own parts for the epilogue's roundings.
"""
import numpy as np
import pytest
import torch

import dash_inputs as di
import matrix_inverse_roots_amd as dash
import mx_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0**-23
FMTS = [dash.DASH_MX_E2M1, dash.DASH_MX_E4M3]
IDS = ["e2m1", "e4m3"]
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def host(t):
    torch.cuda.synchronize()
    return t.detach().cpu()


def f64(t):
    return host(t).double().numpy()


def dev_codes(code, scale, fmt):
    return (torch.from_numpy(ref.pack(code, fmt)).to(DEV).contiguous(),
            torch.from_numpy(scale.astype(np.uint8)).to(DEV).contiguous())


def random_codes(rng, N, rows, cols, fmt, lo=120, hi=134):
    """Every code but NaN, scales 2^-7 .. 2^6, padding zero; (codes, scales, values in 64 bits)."""
    g = -(-cols // 32)
    c = rng.integers(0, 16 if fmt == dash.DASH_MX_E2M1 else 256, (N, rows, g * 32))
    if fmt == dash.DASH_MX_E4M3:
        c[c % 128 == 127] = 0
    c[..., cols:] = 0
    s = rng.integers(lo, hi, (N, rows, g))
    q, b = dev_codes(c, s, fmt)
    return q, b, ref.values(ref.pack(c, fmt), s, cols, fmt)


# ------------------------------------------------------------------------------------------------
# Quantisation
# ------------------------------------------------------------------------------------------------


def hard_matrix(rng, N, rows, cols):
    """Ordinary values, and groups of zeros, of one value, of subnormals, of huge values, near ties and
    borders, with an Inf, with a NaN."""
    x = rng.standard_normal((N, rows, cols)).astype(np.float32) * np.exp2(rng.integers(-8, 9, (N, rows, 1))).astype(np.float32)
    flat = x.reshape(N * rows, cols)
    for r in range(0, N * rows, 9):
        kind = (r // 9) % 8
        w = slice(0, min(cols, 40))
        n = len(range(*w.indices(cols)))
        if kind == 0:
            flat[r, w] = 0
        elif kind == 1:
            flat[r, w] = 1e-40
        elif kind == 2:
            flat[r, w] *= np.float32(1e30)
        elif kind == 3:
            flat[r, w] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -5.0, -2.5, 448.0, 447.9], n)
        elif kind == 4:
            flat[r, 0] = np.inf
        elif kind == 5:
            flat[r, n - 1] = np.nan
        elif kind == 6:
            flat[r, w] = np.nextafter(np.float32(6.0), np.float32(7.0)) if r % 2 else 7.5
        else:
            flat[r, w] = np.float32(3e38)
    return x


SHAPES = [(1, 1, 1), (1, 1, 33), (3, 5, 31), (1, 70, 100), (2, 64, 64), (1, 129, 259), (2, 300, 130), (1, 40, 4100)]


@pytest.mark.parametrize("sides", ["rows", "cols", "both"])
@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
def test_quantize_equals_the_definition(dtype, fmt, sides):
    rng = di.rng(70 + len(sides))
    for N, rows, cols in SHAPES:
        for pad in (0, 8, 3):  # row pitches: as wide as the row, 16-byte aligned or not
            x = torch.from_numpy(hard_matrix(rng, N, rows, cols)).to(dtype)
            buf = torch.full((N, rows, cols + pad), 77.0, dtype=dtype, device=DEV)
            buf[:, :, :cols] = x.to(DEV)
            src = buf[:, :, :cols]
            want = x.double().numpy()
            out = {}
            for side, m in (("rows", want), ("cols", want.transpose(0, 2, 1))):
                if sides in (side, "both"):
                    c, s = dash.mx_buffers(*m.shape, fmt, device=DEV)
                    # a guard behind each buffer
                    c = torch.full((c.numel() + 64,), 0xA5, dtype=torch.uint8, device=DEV)
                    s = torch.full((s.numel() + 64,), 0xA5, dtype=torch.uint8, device=DEV)
                    out[side] = (c, s)
            none = (None, None)
            dash.dash_mx_quantize(src, N, rows, cols, fmt, *out.get("rows", none), *out.get("cols", none))
            for side, m in (("rows", want), ("cols", want.transpose(0, 2, 1))):
                if side in out:
                    c, s = (host(t).numpy() for t in out[side])
                    code, byte = ref.quantize(m, fmt)
                    code = ref.pack(code, fmt).reshape(-1)
                    assert np.array_equal(s[:-64], byte.reshape(-1)), (N, rows, cols, pad, side)
                    assert np.array_equal(c[:-64], code), (N, rows, cols, pad, side)
                    assert np.all(c[-64:] == 0xA5) and np.all(s[-64:] == 0xA5)


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,rows,cols", [(66, 1024, 1024), (1, 8300, 8191)])
def test_quantize_large_stacks(N, rows, cols, fmt):
    """Sizes that take the wide column tiles: as the rows of the matrices and of their transposes."""
    gen = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn((N, rows, cols), generator=gen, device=DEV)
    x *= torch.exp2(torch.randint(-20, 20, (N, rows, 1), generator=gen, device=DEV).float())
    x[0, 5, 7], x[-1, -1, -1] = float("inf"), float("nan")
    both = [dash.mx_buffers(N, rows, cols, fmt, device=DEV), dash.mx_buffers(N, cols, rows, fmt, device=DEV)]
    dash.dash_mx_quantize(x, N, rows, cols, fmt, *both[0], *both[1])
    alone = dash.mx_buffers(N, cols, rows, fmt, device=DEV)
    dash.dash_mx_quantize(x, N, rows, cols, fmt, None, None, *alone)
    for m, got in ((x, both[0]), (x.transpose(1, 2).contiguous(), both[1])):
        want = dash.mx_buffers(*m.shape, fmt, device=DEV)
        dash.dash_mx_quantize(m, *m.shape, fmt, *want)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(alone[0], both[1][0]) and torch.equal(alone[1], both[1][1])
    # and a few rows of it against the definition
    code, byte = ref.quantize(x[0, :9].double().cpu().numpy(), fmt)
    assert np.array_equal(host(both[0][0][0, :9]).numpy(), ref.pack(code, fmt))
    assert np.array_equal(host(both[0][1][0, :9]).numpy(), byte)


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("sides", ["rows", "both"])
def test_quantize_diagonal(fmt, sides):
    rng = di.rng(75)
    for N, B in ((1, 1), (3, 64), (2, 130)):
        x = rng.standard_normal((N, B, B)).astype(np.float32)
        x += 100 * np.eye(B, dtype=np.float32)
        t = torch.from_numpy(x).to(DEV)
        c, s = dash.mx_buffers(N, B, B, fmt, device=DEV)
        ct, st = dash.mx_buffers(N, B, B, fmt, device=DEV) if sides == "both" else (None, None)
        d = torch.empty((N, B), device=DEV)
        dash.dash_mx_quantize(t, N, B, B, fmt, c, s, ct, st, diag=d)
        off = x * (1 - np.eye(B))
        assert np.array_equal(host(d).numpy(), np.diagonal(x, axis1=1, axis2=2))
        for codes, scales, m in ((c, s, off), (ct, st, off.transpose(0, 2, 1))):
            if codes is None:
                continue
            code, byte = ref.quantize(m, fmt)
            assert np.array_equal(host(scales).numpy(), byte)
            assert np.array_equal(host(codes).numpy(), ref.pack(code, fmt))
        v = torch.empty((N, B, B), device=DEV)
        dash.dash_mx_dequantize(c, s, N, B, B, fmt, v, diag=d)
        code, byte = ref.quantize(off, fmt)
        want = ref.values(ref.pack(code, fmt), byte, B, fmt) + x * np.eye(B)
        assert np.array_equal(f64(v), want)


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
def test_dequantize_every_code_and_scale(dtype, fmt):
    codes = np.arange(16 if fmt == dash.DASH_MX_E2M1 else 256)
    cols = len(codes)
    code = np.zeros((256, -(-cols // 32) * 32), np.int64)
    code[:, :cols] = codes
    byte = np.repeat(np.arange(256)[:, None], code.shape[1] // 32, 1)
    c, s = dev_codes(code, byte, fmt)
    buf = torch.full((256, cols + 5), 7.0, dtype=dtype, device=DEV)
    dash.dash_mx_dequantize(c, s, 1, 256, cols, fmt, buf[:, :cols])
    want = torch.from_numpy(ref.values(ref.pack(code, fmt), byte, cols, fmt))
    # every value is an fp32 number: one rounding to the type
    want = want.float().to(dtype)
    got = host(buf)
    assert torch.equal(torch.isnan(got[:, :cols]), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got[:, :cols], nan=0.0), torch.nan_to_num(want, nan=0.0))
    assert bool((got[:, cols:] == 7.0).all())


def test_quantize_past_32_bit_offsets():
    """More than 2^32 elements: the last rows are as a small call makes them."""
    rows, cols = (1 << 19) + 3, 8200
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV).fill_(1.0)
    tail = torch.randn((5, cols), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    x[-5:] = tail.to(torch.bfloat16)
    fmt = dash.DASH_MX_E4M3
    c, s = dash.mx_buffers(1, rows, cols, fmt, device=DEV)
    ct, st = dash.mx_buffers(1, cols, rows, fmt, device=DEV)
    dash.dash_mx_quantize(x, 1, rows, cols, fmt, c, s)
    c5, s5 = dash.mx_buffers(1, 5, cols, fmt, device=DEV)
    dash.dash_mx_quantize(x[-5:], 1, 5, cols, fmt, c5, s5)
    assert torch.equal(c[0, -5:], c5[0]) and torch.equal(s[0, -5:], s5[0])
    c2, s2 = torch.zeros_like(c), torch.zeros_like(s)
    dash.dash_mx_quantize(x, 1, rows, cols, fmt, c2, s2, ct, st)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    c3 = torch.zeros((1, 3, ct.shape[2]), dtype=torch.uint8, device=DEV)
    s3 = torch.zeros((1, 3, st.shape[2]), dtype=torch.uint8, device=DEV)
    dash.dash_mx_quantize(x[:, -3:].t().contiguous(), 1, 3, rows, fmt, c3, s3)
    assert torch.equal(ct[0, -3:], c3[0]) and torch.equal(st[0, -3:], s3[0])
    v = torch.empty_like(x)
    dash.dash_mx_dequantize(c, s, 1, rows, cols, fmt, v)
    v5 = torch.empty_like(x[-5:])
    dash.dash_mx_dequantize(c5, s5, 1, 5, cols, fmt, v5)
    assert torch.equal(v[-5:], v5) and bool((v[:-5] == 1.0).all())


# ------------------------------------------------------------------------------------------------
# Statistics
# ------------------------------------------------------------------------------------------------


def stats_want(q, qt, A, beta):
    """(new statistics, bound) in 64 bits"""
    N, B = q.shape[0], q.shape[1]
    g = np.concatenate((q, qt))
    S = g @ g.transpose(0, 2, 1)
    mag = np.abs(g) @ np.abs(g).transpose(0, 2, 1)
    Au = np.triu(A)
    A = Au + np.triu(A, 1).transpose(0, 2, 1)
    want = beta * A + (1 - beta) * S
    return want, (1 - beta) * B * U * mag + 4 * U * (np.abs(beta * A) + (1 - beta) * mag)


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("B", [64, 128, 192, 256, 320, 448, 512])
def test_stats(B, fmt):
    rng = di.rng(80 + B)
    for N, beta in ((1, 0.95), (3, 0.5)) if B < 512 else ((2, 0.9),):
        q, s, v = random_codes(rng, N, B, B, fmt)
        qt, st, vt = random_codes(rng, N, B, B, fmt)
        A = rng.standard_normal((2 * N, B, B)).astype(np.float32) * 100
        Ad = torch.from_numpy(A).to(DEV)
        low = torch.tril(torch.ones((B, B), dtype=torch.bool, device=DEV), -1)
        Ad[:, low] = float("nan")  # the lower triangle is not read
        b32 = float(np.float32(beta))
        dash.dash_update_stats_mx(q, s, qt, st, N, B, fmt, beta, Ad)
        got = f64(Ad)
        want, tol = stats_want(v, vt, A.astype(np.float64), b32)
        assert np.all(np.abs(got - want) <= tol), (N, np.max(np.abs(got - want) / tol))
        assert np.array_equal(got, got.transpose(0, 2, 1))


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
def test_stats_edges(fmt):
    N, B = 2, 128
    rng = di.rng(90)
    q, s, v = random_codes(rng, N, B, B, fmt)
    A = torch.zeros((2 * N, B, B), device=DEV)
    # beta = 1 keeps A, beta = 0 drops a finite A
    A[:, 3, 5] = A[:, 5, 3] = 2.5
    dash.dash_update_stats_mx(q, s, q, s, N, B, fmt, 1.0, A)
    want = torch.zeros_like(A)
    want[:, 3, 5] = want[:, 5, 3] = 2.5
    assert torch.equal(A, want)
    dash.dash_update_stats_mx(q, s, q, s, N, B, fmt, 0.0, A)
    w, tol = stats_want(v, v, np.zeros((2 * N, B, B)), 0.0)
    assert np.all(np.abs(f64(A) - w) <= tol)
    # one NaN group of tile 1, row 7: that row and column of L_1, nothing else
    s2 = s.clone()
    s2[1, 7, 2] = 255
    q2 = q.clone()
    w = q.shape[2] // 4
    q2[1, 7, 2 * w:3 * w] = 0
    A = torch.ones((2 * N, B, B), device=DEV)
    dash.dash_update_stats_mx(q2, s2, q, s, N, B, fmt, 0.5, A)
    bad = torch.isnan(A)
    want = torch.zeros_like(bad)
    want[1, 7, :] = want[1, :, 7] = True
    assert torch.equal(bad, want)
    # small whole numbers: exact
    one = torch.full_like(s, 127)
    c = rng.integers(0, 3, (N, B, B)) * 2 if fmt == dash.DASH_MX_E2M1 else rng.integers(0, 2, (N, B, B)) * 0x38
    qc, _ = dev_codes(c, np.full((N, B, B // 32), 127), fmt)
    vc = ref.values(ref.pack(c, fmt), np.full((N, B, B // 32), 127), B, fmt)
    A = torch.zeros((2 * N, B, B), device=DEV)
    dash.dash_update_stats_mx(qc, one, qc, one, N, B, fmt, 0.5, A)
    assert np.array_equal(f64(A)[:N], 0.5 * (vc @ vc.transpose(0, 2, 1)))


# ------------------------------------------------------------------------------------------------
# Update
# ------------------------------------------------------------------------------------------------


def apply_want(L, R, G):
    """(L G R^T, bound): T = L G is off by K U |L||G| and rounded, then the second product's own sum."""
    B = G.shape[1]
    Rt = R.transpose(0, 2, 1)
    mag = np.abs(L) @ np.abs(G) @ np.abs(Rt)
    return L @ G @ Rt, 2 * (B + 4) * U * mag


@pytest.mark.parametrize("diag", [False, True])
@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("B", [64, 128, 192, 256, 320, 512])
def test_apply(B, fmt, diag):
    rng = di.rng(100 + B)
    N = 3 if B < 512 else 1
    ql, sl, L = random_codes(rng, N, B, B, fmt)
    qr, sr, R = random_codes(rng, N, B, B, fmt)
    dl = dr = None
    if diag:
        dl, dr = (torch.from_numpy(rng.standard_normal((N, B)).astype(np.float32) * 50).to(DEV) for _ in range(2))
        L = L + f64(dl)[:, :, None] * np.eye(B)
        R = R + f64(dr)[:, :, None] * np.eye(B)
    G = rng.standard_normal((N, B, B)).astype(np.float32) * np.float32(1e-3)
    Gd = torch.from_numpy(G).to(DEV)
    Ud = torch.full((N, B, B), float("nan"), device=DEV)
    ws = dash.workspace(dash.DASH_OP_APPLY, N, B, device=DEV)
    ws.fill_(0xFF)
    dash.dash_apply_mx(ql, sl, qr, sr, Gd, N, B, fmt, Ud, XL_diag=dl, XR_diag=dr, ws=ws)
    want, tol = apply_want(L, R, G.astype(np.float64))
    err = np.abs(f64(Ud) - want)
    assert np.all(err <= tol), np.max(err / tol)
    # as near to 64 bits as an fp32 product: 2^-24 sqrt(K) or so, far inside the bound above
    assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(want)
    assert np.array_equal(f64(Gd), G.astype(np.float64))


@pytest.mark.parametrize("diag", [False, True])
@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("N,B", [(500, 64), (300, 128), (60, 256), (50, 320), (40, 448), (130, 512)])
def test_apply_wide(N, B, fmt, diag):
    """Stacks that take 128- and 256-wide kernel tiles, whole and at the edges."""
    rng = di.rng(110 + B)
    ql, sl, L = random_codes(rng, N, B, B, fmt)
    qr, sr, R = random_codes(rng, N, B, B, fmt)
    L, R = torch.from_numpy(L).to(DEV), torch.from_numpy(R).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(B)
    dl = dr = None
    if diag:
        dl, dr = (50 * torch.randn((N, B), generator=gen, device=DEV) for _ in range(2))
        L, R = L + torch.diag_embed(dl.double()), R + torch.diag_embed(dr.double())
    G = torch.randn((N, B, B), generator=gen, device=DEV)
    G *= torch.logspace(-6, 6, N, device=DEV)[:, None, None]  # blocks of their own magnitudes
    got = torch.full((N, B, B), float("nan"), device=DEV)
    ws = dash.workspace(dash.DASH_OP_APPLY, N, B, device=DEV)
    ws.fill_(0xFF)
    dash.dash_apply_mx(ql, sl, qr, sr, G, N, B, fmt, got, XL_diag=dl, XR_diag=dr, ws=ws)
    Rt = R.transpose(1, 2).contiguous()
    want = torch.bmm(torch.bmm(L, G.double()), Rt)
    mag = torch.bmm(torch.bmm(L.abs(), G.double().abs()), Rt.abs())
    err = (got.double() - want).abs()
    assert bool((err <= 2 * (B + 4) * U * mag).all())
    rel = err.flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    assert float(rel.max()) <= 2e-6
    # each block as a call of its own makes it, to the products' rounding
    one = torch.empty((1, B, B), device=DEV)
    i = N // 2
    dash.dash_apply_mx(ql[i:i + 1], sl[i:i + 1], qr[i:i + 1], sr[i:i + 1], G[i:i + 1], 1, B, fmt, one,
                       XL_diag=dl[i:i + 1] if diag else None, XR_diag=dr[i:i + 1] if diag else None, ws=ws)
    assert bool(((one[0].double() - want[i]).abs() <= 2 * (B + 4) * U * mag[i]).all())


def test_apply_identity_and_ranges():
    """Unit roots give G back bit for bit; blocks of very different magnitudes do not touch each other."""
    fmt, N, B = dash.DASH_MX_E2M1, 4, 192
    q, s = dash.mx_buffers(N, B, B, fmt, device=DEV)
    q.zero_()
    s.fill_(127)
    d = torch.ones((N, B), device=DEV)
    rng = di.rng(120)
    G = torch.from_numpy(rng.standard_normal((N, B, B)).astype(np.float32)).to(DEV)
    G *= torch.tensor([1.0, 1e-30, 1e25, 1e-12], device=DEV)[:, None, None]
    Ud = torch.empty_like(G)
    ws = dash.workspace(dash.DASH_OP_APPLY, N, B, device=DEV)
    dash.dash_apply_mx(q, s, q, s, G, N, B, fmt, Ud, XL_diag=d, XR_diag=d, ws=ws)
    assert torch.equal(Ud, G)
    # a diagonal held in the codes instead: 1.0 is E2M1 code 2
    c = np.zeros((N, B, B), np.int64)
    c[:, np.arange(B), np.arange(B)] = 2
    q, s = dev_codes(c, np.full((N, B, B // 32), 127), fmt)
    dash.dash_apply_mx(q, s, q, s, G, N, B, fmt, Ud, ws=ws)
    g = f64(G)
    # (binary16 pieces hold 22 bits of the block's largest elements)
    assert np.all(np.abs(f64(Ud) - g) <= 2.0**-21 * np.abs(g).max(axis=(1, 2), keepdims=True))
    # a NaN in one block's G stays in that block
    G2 = G.clone()
    G2[2, 5, 6] = float("nan")
    dash.dash_apply_mx(q, s, q, s, G2, N, B, fmt, Ud, ws=ws)
    bad = torch.isnan(Ud).flatten(1).any(1).cpu().tolist()
    assert bad == [False, False, True, False]


# ------------------------------------------------------------------------------------------------
# Gradient tiles
# ------------------------------------------------------------------------------------------------


def grad(dY, q, s, fmt, T, out, inp, B, accumulate=False, G=None, guard=0):
    n = -(-out // B) * -(-inp // B) * B * B
    buf = torch.full((n + guard,), float("nan"), device=DEV) if G is None else G
    ws = dash.grad_stack_mx_workspace(T, out, inp, dY.dtype, device=DEV)
    if ws is not None:
        ws.fill_(0xFF)
    dash.dash_grad_stack_mx(dY, q, s, fmt, T, out, inp, B, buf, accumulate=accumulate, ws=ws)
    return buf


GRADS = [(1, 1, 1, 64), (1, 64, 64, 64), (31, 70, 33, 64), (32, 256, 256, 128), (33, 257, 300, 128), (100, 64, 500, 256),
         (257, 130, 64, 192), (64, 600, 520, 192), (1500, 72, 40, 64), (5000, 300, 129, 256), (2600, 520, 264, 2048)]


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
def test_grad_stack(dtype, fmt):
    rng = di.rng(130)
    for T, out, inp, B in GRADS:
        q, s, X = random_codes(rng, 1, T, inp, fmt)
        for pad in (0, 8, 3):
            buf = torch.full((T, out + pad), float("nan"), dtype=dtype, device=DEV)  # beyond the columns: not read
            buf[:, :out] = torch.from_numpy(rng.standard_normal((T, out))).to(DEV).to(dtype)
            dY = buf[:, :out]
            d = f64(dY)
            W, mag = d.T @ X[0], np.abs(d).T @ np.abs(X[0])
            # piece products: up to three addends for a term, splits joined in a further sum of up to 256
            tol = ref.tiles((3 * T + 260) * U * mag, B)
            G = grad(dY, q, s, fmt, T, out, inp, B, guard=64)
            got = f64(G)
            assert np.all(np.isnan(got[-64:]))
            got = got[:-64].reshape(-1, B, B)
            want = ref.tiles(W, B)
            err = np.abs(got - want)
            assert np.all(err <= tol), (T, out, inp, B, pad, np.nanmax(err - tol))
            assert np.linalg.norm(err) <= 3e-6 * np.linalg.norm(mag)
            again = grad(dY, q, s, fmt, T, out, inp, B, guard=64)
            assert torch.equal(again[:-64], G[:-64])  # equal calls, equal bits


# tokens, out, in, B that take 128- and 256-wide kernel tiles, whole and at the edges, split and not
WIDE_GRADS = [(200, 2070, 7000, 512), (90, 3000, 2100, 256), (7000, 600, 520, 192), (4100, 2050, 2048, 1024)]


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,out,inp,B", WIDE_GRADS)
def test_grad_stack_wide(T, out, inp, B, dtype):
    fmt = dash.DASH_MX_E4M3 if T % 200 else dash.DASH_MX_E2M1
    rng = di.rng(135 + T)
    q, s, X = random_codes(rng, 1, T, inp, fmt)
    Xd = torch.from_numpy(X[0]).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(T)
    for pad in (0, 6):
        buf = torch.full((T, out + pad), float("nan"), dtype=dtype, device=DEV)
        buf[:, :out] = torch.randn((T, out), generator=gen, device=DEV).to(dtype)
        dY = buf[:, :out]
        d = dY.double()
        W, mag = (d.T.contiguous() @ Xd).cpu().numpy(), (d.abs().T.contiguous() @ Xd.abs()).cpu().numpy()
        tol = ref.tiles((3 * T + 260) * U * mag, B)
        G = grad(dY, q, s, fmt, T, out, inp, B)
        err = np.abs(f64(G).reshape(-1, B, B) - ref.tiles(W, B))
        assert np.all(err <= tol), (pad, np.nanmax(err - tol))
        assert np.linalg.norm(err) <= 3e-6 * np.linalg.norm(mag)
        assert torch.equal(grad(dY, q, s, fmt, T, out, inp, B), G)
        old = torch.randn(G.shape, generator=gen, device=DEV)
        more = grad(dY, q, s, fmt, T, out, inp, B, True, old.clone())
        assert torch.equal(more, old + G)  # one fp32 addition of the same sum


@pytest.mark.parametrize("T", [0, 1, 40, 3000])
def test_grad_stack_accumulates(T):
    fmt, out, inp, B = dash.DASH_MX_E4M3, 100, 70, 64
    rng = di.rng(140 + T)
    q, s, X = random_codes(rng, 1, T, inp, fmt)
    dY = torch.from_numpy(rng.standard_normal((T, out)).astype(np.float32)).to(DEV)
    old = torch.from_numpy(rng.standard_normal((4, B, B)).astype(np.float32)).to(DEV)
    got = grad(dY, q, s, fmt, T, out, inp, B, True, old.clone())
    W, mag = f64(dY).T @ X[0], np.abs(f64(dY)).T @ np.abs(X[0])
    want = f64(old) + ref.tiles(W, B)
    tol = ref.tiles((3 * T + 260) * U * mag, B) + U * np.abs(want)
    assert np.all(np.abs(f64(got) - want) <= tol)
    # without it the tiles' old values do not matter, and an empty sum is zero
    fresh = grad(dY, q, s, fmt, T, out, inp, B)
    assert bool(torch.isfinite(fresh).all())
    if T == 0:
        assert torch.equal(got, old) and not fresh.any()
        dash.dash_grad_stack_mx(None, None, None, fmt, 0, out, inp, B, old, ldy=out, stream=0)
        assert not old.any()


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
def test_grad_stack_nonfinite_rows(dtype):
    """A NaN group and an Inf in dY reach their own row and column of the weight only."""
    fmt, T, out, inp, B = dash.DASH_MX_E4M3, 70, 96, 96, 128
    rng = di.rng(150)
    q, s, X = random_codes(rng, 1, T, inp, fmt)
    q[0, 11, 32:64] = 0
    s[0, 11, 1] = 255
    dY = torch.from_numpy(rng.standard_normal((T, out))).to(DEV).to(dtype)
    dY[20, 9] = float("inf")
    G = f64(grad(dY, q, s, fmt, T, out, inp, B)).reshape(B, B)
    bad = np.zeros((B, B), bool)
    bad[:out, 32:64] = True
    bad[9, :inp] = True
    assert np.array_equal(~np.isfinite(G), bad)


@pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
def test_unaligned_views(dtype):
    """Views that start on their element only, at every offset within 16 bytes: as their aligned copies."""
    fmt, T, out, inp, B = dash.DASH_MX_E4M3, 130, 300, 77, 128
    rng = di.rng(155)
    q, s, _ = random_codes(rng, 1, T, inp, fmt)
    buf = torch.from_numpy(rng.standard_normal((T, out + 24))).to(DEV).to(dtype)
    for shift in range(1, 9):
        view = buf[:, shift:shift + out]
        copy = torch.empty((T, out + 12), dtype=dtype, device=DEV)[:, :out]  # rows of another pitch
        copy.copy_(view)
        assert torch.equal(grad(view, q, s, fmt, T, out, inp, B), grad(copy, q, s, fmt, T, out, inp, B))
        for sides in (("rows",), ("cols",), ("rows", "cols")):
            got = []
            for src in (view, copy.contiguous()):
                pair = [dash.mx_buffers(1, T, out, fmt, device=DEV), dash.mx_buffers(1, out, T, fmt, device=DEV)]
                args = [x if side in sides else (None, None) for side, x in zip(("rows", "cols"), pair)]
                dash.dash_mx_quantize(src, 1, T, out, fmt, *args[0], *args[1])
                got.append([x for a in args for x in a if x is not None])
            assert all(torch.equal(x, y) for x, y in zip(*got))
        c, sc = dash.mx_buffers(1, T, out, fmt, device=DEV)
        dash.dash_mx_quantize(view, 1, T, out, fmt, c, sc)
        back, wide = torch.zeros_like(buf), torch.empty((T, out), dtype=dtype, device=DEV)
        dash.dash_mx_dequantize(c, sc, 1, T, out, fmt, back[:, shift:shift + out])
        dash.dash_mx_dequantize(c, sc, 1, T, out, fmt, wide)
        assert torch.equal(back[:, shift:shift + out], wide)
        assert not back[:, :shift].any() and not back[:, shift + out:].any()


def test_grad_stack_past_32_bit_offsets():
    """Rows of dY beyond 2^31 elements, codes beyond 2^32 bytes."""
    fmt = dash.DASH_MX_E4M3
    T, ldy, out, inp, B = 70001, 32776, 40, 62016, 64
    dY = torch.zeros((T, ldy), dtype=torch.bfloat16, device=DEV)[:, :out]
    q, s = dash.mx_buffers(1, T, inp, fmt, device=DEV)
    q.zero_()
    s.fill_(127)
    dY[-1, 3] = 2.0
    dY[-2, 7] = -1.0
    q[0, -1, inp - 1] = 0x38  # 1.0
    q[0, -2, 100] = 0x40  # 2.0
    G = grad(dY, q, s, fmt, T, out, inp, B).reshape(-1, B, B)
    assert int(torch.count_nonzero(G)) == 2
    assert float(G[(inp - 1) // B, 3, (inp - 1) % B]) == 2.0 and float(G[1, 7, 100 - 64]) == -2.0


def test_grad_stack_against_differences():
    """f(W) = sum tanh(Q W^T)^2 / 2 in 64 bits: central differences in single weights against the tiles."""
    fmt, T, out, inp, B = dash.DASH_MX_E4M3, 90, 40, 72, 64
    rng = di.rng(160)
    x = torch.from_numpy(rng.standard_normal((T, inp)).astype(np.float32)).to(DEV)
    q, s = dash.mx_buffers(1, T, inp, fmt, device=DEV)
    dash.dash_mx_quantize(x, 1, T, inp, fmt, q, s)
    X = ref.values(host(q).numpy(), host(s).numpy(), inp, fmt)[0]
    W = rng.standard_normal((out, inp)) * 0.2

    def f(w):
        return 0.5 * np.sum(np.tanh(X @ w.T) ** 2)

    y = np.tanh(X @ W.T)
    dY = torch.from_numpy((y * (1 - y * y)).astype(np.float32)).to(DEV)
    G = f64(grad(dY, q, s, fmt, T, out, inp, B)).reshape(1, 2, B, B)
    for i, j in ((0, 0), (3, 70), (39, 71), (20, 33), (7, 64)):
        h = 1e-4
        E = np.zeros_like(W)
        E[i, j] = h
        d = (f(W + E) - f(W - E)) / (2 * h)
        # h^2 f''' / 6 with |x| <= 4: 1e-8 T 64; rounding of f at 2^-53 / h; dY and sums in fp32
        assert abs(G[0, j // B, i, j % B] - d) <= 1e-5 + 1e-5 * abs(d), (i, j)


# ------------------------------------------------------------------------------------------------
# Together
# ------------------------------------------------------------------------------------------------


def pipeline(x, dY, fmt8, fmt4, out, inp, B, buf):
    """One layer's step: 8-bit checkpoint -> gradient tiles -> statistics -> roots in 4 bits -> update."""
    T = x.shape[0]
    N = -(-out // B) * -(-inp // B)
    b = buf
    dash.dash_mx_quantize(x, 1, T, inp, fmt8, b["x"], b["xs"])
    dash.dash_grad_stack_mx(dY, b["x"], b["xs"], fmt8, T, out, inp, B, b["G"], ws=b["gws"])
    dash.dash_mx_quantize(b["G"], N, B, B, fmt8, b["g"], b["gs"], b["gt"], b["gts"])
    dash.dash_update_stats_mx(b["g"], b["gs"], b["gt"], b["gts"], N, B, fmt8, 0.5, b["A"])
    dash.dash_scale(b["A"], 2 * N, B, dash.DASH_SCALE_FROBENIUS, dash.DASH_FP32, 0, 0, None, b["s"], None)
    dash.dash_inverse_root_ndb(b["A"], b["s"], 2 * N, B, 14, 14, b["X"], status=b["st"], ws=b["nws"])
    dash.dash_mx_quantize(b["X"], 2 * N, B, B, fmt4, b["r"], b["rs"], diag=b["d"])
    dash.dash_apply_mx(b["r"][:N], b["rs"][:N], b["r"][N:], b["rs"][N:], b["G"], N, B, fmt4, b["U"], XL_diag=b["d"][:N],
                       XR_diag=b["d"][N:], ws=b["aws"])
    dash.dash_unstack(b["U"], B, [b["W"]])


def pipeline_buffers(T, fmt8, fmt4, out, inp, B):
    N = -(-out // B) * -(-inp // B)
    b = {}
    b["x"], b["xs"] = dash.mx_buffers(1, T, inp, fmt8, device=DEV)
    b["G"], b["U"] = torch.empty((N, B, B), device=DEV), torch.empty((N, B, B), device=DEV)
    b["gws"] = dash.grad_stack_mx_workspace(T, out, inp, torch.bfloat16, device=DEV)
    b["g"], b["gs"] = dash.mx_buffers(N, B, B, fmt8, device=DEV)
    b["gt"], b["gts"] = dash.mx_buffers(N, B, B, fmt8, device=DEV)
    b["A"] = (torch.eye(B, device=DEV) * 40.0).expand(2 * N, B, B).contiguous()
    b["s"], b["st"] = torch.empty(2 * N, device=DEV), torch.empty(2 * N, dtype=torch.int32, device=DEV)
    b["X"] = torch.empty((2 * N, B, B), device=DEV)
    b["nws"] = dash.workspace(dash.DASH_OP_NDB, 2 * N, B, device=DEV)
    b["r"], b["rs"] = dash.mx_buffers(2 * N, B, B, fmt4, device=DEV)
    b["d"] = torch.empty((2 * N, B), device=DEV)
    b["aws"] = dash.workspace(dash.DASH_OP_APPLY, N, B, device=DEV)
    b["W"] = torch.empty((out, -(-inp // 4) * 4), device=DEV)[:, :inp]
    return b


def pipeline_inputs(seed, T, out, inp):
    rng = di.rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, inp))).to(DEV).to(torch.bfloat16)
    dY = torch.from_numpy(rng.standard_normal((T, -(-out // 8) * 8)) * 0.1).to(DEV).to(torch.bfloat16)[:, :out]
    return x, dY


def test_the_operators_together():
    """Each stage against 64-bit arithmetic on what the stage before it left."""
    fmt8, fmt4 = dash.DASH_MX_E4M3, dash.DASH_MX_E2M1
    T, out, inp, B = 700, 150, 200, 128
    x, dY = pipeline_inputs(170, T, out, inp)
    b = pipeline_buffers(T, fmt8, fmt4, out, inp, B)
    A0 = f64(b["A"])
    pipeline(x, dY, fmt8, fmt4, out, inp, B, b)
    code, byte = ref.quantize(f64(x)[None], fmt8)
    assert np.array_equal(host(b["x"]).numpy(), ref.pack(code, fmt8))
    X = ref.values(ref.pack(code, fmt8), byte, inp, fmt8)[0]
    G = f64(b["G"])
    mag = np.abs(f64(dY)).T @ np.abs(X)
    assert np.all(np.abs(G - ref.tiles(f64(dY).T @ X, B)) <= ref.tiles((T + 260) * U * mag, B))
    parts = []
    for m in (G, G.transpose(0, 2, 1)):
        code, byte = ref.quantize(m, fmt8)
        parts.append(ref.values(ref.pack(code, fmt8), byte, B, fmt8))
    want, tol = stats_want(parts[0], parts[1], A0, 0.5)
    assert np.all(np.abs(f64(b["A"]) - want) <= tol)
    assert not host(b["st"]).any()
    Xr = f64(b["X"])
    eye = np.eye(B)
    code, byte = ref.quantize(Xr * (1 - eye), fmt4)
    R = ref.values(ref.pack(code, fmt4), byte, B, fmt4) + Xr * eye
    N = G.shape[0]
    want, tol = apply_want(R[:N], R[N:], G)
    assert np.all(np.abs(f64(b["U"]) - want) <= tol)
    # 4-bit roots with their own diagonals stay near the fp32 update
    full = Xr[:N] @ G @ Xr[N:]
    assert np.linalg.norm(want - full) <= 0.15 * np.linalg.norm(full)
    W = f64(b["W"])
    assert np.array_equal(ref.tiles(W, B)[0], f64(b["U"])[0])


def test_side_stream_equals_default():
    fmt8, fmt4 = dash.DASH_MX_E4M3, dash.DASH_MX_E2M1
    T, out, inp, B = 3000, 150, 200, 128  # (the token axis is split)
    x, dY = pipeline_inputs(171, T, out, inp)
    b1, b2 = (pipeline_buffers(T, fmt8, fmt4, out, inp, B) for _ in range(2))
    pipeline(x, dY, fmt8, fmt4, out, inp, B, b1)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        pipeline(x, dY, fmt8, fmt4, out, inp, B, b2)
    torch.cuda.synchronize()
    for k in ("x", "G", "g", "gt", "A", "r", "d", "U"):
        assert torch.equal(b1[k], b2[k]), k


def test_captured_step_replays():
    """The quantise, gradient, statistics and update calls in a captured graph: every replay on new inputs
    equals the eager calls."""
    fmt8, fmt4 = dash.DASH_MX_E4M3, dash.DASH_MX_E2M1
    T, out, inp, B = 3000, 150, 200, 128
    x, dY = pipeline_inputs(172, T, out, inp)
    b, e = (pipeline_buffers(T, fmt8, fmt4, out, inp, B) for _ in range(2))
    pipeline(x, dY, fmt8, fmt4, out, inp, B, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pipeline(x, dY, fmt8, fmt4, out, inp, B, b)
    for seed in (173, 174, 175):
        x2, dY2 = pipeline_inputs(seed, T, out, inp)
        x.copy_(x2)
        dY.copy_(dY2)
        b["A"].copy_(e["A"])
        g.replay()
        torch.cuda.synchronize()
        pipeline(x2, dY2, fmt8, fmt4, out, inp, B, e)
        torch.cuda.synchronize()
        for k in ("x", "G", "g", "gt", "A", "r", "d", "U"):
            assert torch.equal(b[k], e[k]), (seed, k)


@pytest.mark.parametrize("B", [64, 128, 192, 320, 448])
@pytest.mark.parametrize("N", [1, 50])
def test_nothing_is_written_past_the_buffers(N, B):
    """Outputs and exactly sized workspaces end where they say, for every tile width and edge."""
    fmt8, fmt4 = dash.DASH_MX_E4M3, dash.DASH_MX_E2M1
    rng = di.rng(180 + B)

    def guarded(n, dtype=torch.float32):
        buf = torch.full((n + 4096,), 77, dtype=dtype, device=DEV)
        return buf, buf[:n]

    tails = []
    for fmt in (fmt8, fmt4):
        q, s, _ = random_codes(rng, 1, B, B, fmt)
        q, s = q.expand(N, -1, -1).contiguous(), s.expand(N, -1, -1).contiguous()
        G = torch.randn((N, B, B), generator=torch.Generator(device=DEV).manual_seed(B), device=DEV)
        buf, Ud = guarded(N * B * B)
        wbuf, ws = guarded(dash.dash_workspace_size(dash.DASH_OP_APPLY, N, B), torch.uint8)
        dash.dash_apply_mx(q, s, q, s, G, N, B, fmt, Ud, ws=ws)
        tails += [buf[N * B * B:], wbuf[ws.numel():]]
        assert bool(torch.isfinite(Ud).all())
        buf, A = guarded(2 * N * B * B)
        A.zero_()
        dash.dash_update_stats_mx(q, s, q, s, N, B, fmt, 0.5, A)
        tails.append(buf[2 * N * B * B:])
        T, out, inp = 40 * N + 700, B + 9, B - 5
        x, xs, _ = random_codes(rng, 1, T, inp, fmt)
        n = 4 * B * B if inp > B else 2 * B * B
        buf, Gd = guarded(n)
        for dtype in TYPES:
            dY = torch.ones((T, out), dtype=dtype, device=DEV)
            need = dash.dash_grad_stack_mx_workspace(T, out, inp, dash._lib._prec_of(dtype))
            wbuf, ws = guarded(need, torch.uint8)
            dash.dash_grad_stack_mx(dY, x, xs, fmt, T, out, inp, B, Gd, ws=ws if need else None)
            tails += [buf[n:], wbuf[need:]]
    torch.cuda.synchronize()
    for tail in tails:
        assert bool((tail == 77).all())


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own buffers, equal the same calls in turn."""
    fmt8, fmt4 = dash.DASH_MX_E4M3, dash.DASH_MX_E2M1
    T, out, inp, B = 3000, 300, 400, 128
    data = [pipeline_inputs(190 + i, T, out, inp) for i in range(2)]
    ref_b, b = ([pipeline_buffers(T, fmt8, fmt4, out, inp, B) for _ in range(2)] for _ in range(2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        pipeline(*data[i], fmt8, fmt4, out, inp, B, ref_b[i])
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            b[i]["A"].copy_((torch.eye(B, device=DEV) * 40.0).expand_as(b[i]["A"]))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                pipeline(*data[i], fmt8, fmt4, out, inp, B, b[i])
        torch.cuda.synchronize()
        for i in range(2):
            for k in ("x", "G", "g", "gt", "A", "r", "d", "U"):
                assert torch.equal(b[i][k], ref_b[i][k]), (i, k)


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn: each equals its eager call every time."""
    fmt, B = dash.DASH_MX_E4M3, 64
    rng = di.rng(195)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    calls = []
    for T, out, inp in ((5000, 72, 40), (3000, 100, 130)):
        q, s, _ = random_codes(rng, 1, T, inp, fmt)
        dY = torch.from_numpy(rng.standard_normal((T, out)).astype(np.float32)).to(DEV)
        assert 0 < dash.dash_grad_stack_mx_workspace(T, out, inp, dash.DASH_FP32) <= ws.numel()
        G = torch.empty((-(-out // B) * -(-inp // B), B, B), device=DEV)
        calls.append((lambda dY=dY, q=q, s=s, T=T, out=out, inp=inp, G=G: dash.dash_grad_stack_mx(
            dY, q, s, fmt, T, out, inp, B, G, ws=ws), G, dY))
    graphs = []
    for call, G, _ in calls:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for i in range(4):
        for (call, G, dY), g in zip(calls, graphs):
            dY.mul_(-0.5)
            G.fill_(float("nan"))
            g.replay()
            got = G.clone()
            call()
            torch.cuda.synchronize()
            assert torch.equal(G, got), i


def test_wrong_tensors_are_refused():
    x = torch.zeros((64, 64), device=DEV)
    c, s = dash.mx_buffers(1, 64, 64, dash.DASH_MX_E4M3, device=DEV)
    f = dash.dash_mx_quantize
    for bad in (x.t()[:, ::2], x.double(), x[:, :32], x[:32]):
        with pytest.raises(ValueError):
            f(bad, 1, 64, 64, dash.DASH_MX_E4M3, c, s)
    with pytest.raises(ValueError):
        f(x, 1, 64, 64, dash.DASH_MX_E4M3, c[:, :32], s)  # too few codes
    with pytest.raises(ValueError):
        f(x, 1, 64, 64, dash.DASH_MX_E4M3, c, s[:, :, :1].contiguous())
    with pytest.raises(ValueError):
        f(x, 1, 64, 64, dash.DASH_MX_E4M3, c.int(), s)
    with pytest.raises(ValueError):
        f(x.expand(2, 64, 64), 2, 64, 64, dash.DASH_MX_E4M3, *dash.mx_buffers(2, 64, 64, dash.DASH_MX_E4M3, device=DEV))
    G = torch.zeros((1, 64, 64), device=DEV)
    with pytest.raises(ValueError):
        dash.dash_grad_stack_mx(x, c, s, dash.DASH_MX_E4M3, 64, 65, 64, 64, G)
    with pytest.raises(ValueError):
        dash.dash_grad_stack_mx(x, c, s, dash.DASH_MX_E4M3, 64, 64, 64, 128, G)  # the stack is too small
