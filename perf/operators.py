"""Cases and plain forms of the microscaled operators: quantisation, Shampoo statistics from
microscaled gradients, the preconditioned update with microscaled roots, and gradient tiles from a
layer's 8-bit activation checkpoint.

A microscaled row is cut into groups of 32 elements that share a power of two 2^e, held as one byte
e + 127 (255: the group held an Inf or a NaN); an element is an E2M1 (4 bits, two to a byte, the even
one in the low half) or an E4M3 value (8 bits).  e is the least integer with max|x| <= m 2^e, m the
format's largest value (6 or 448), at least -127; elements round to nearest, ties to even.

`run` computes the plain form (elementary torch operations in 32 bits) unless `own` is set, and
calls the library then.  `exact` is the same in 64 bits, written from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32
TOP = {"e2m1": 6.0, "e4m3": 448.0}
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FMTS = ("e2m1", "e4m3")


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------


def _quantize(N, rows, cols, type, fmt, sides, diag=False, **more):
    return {"op": "quantize", "N": N, "rows": rows, "cols": cols, "type": type, "fmt": fmt, "sides": sides,
            "diag": diag, **more}


def _stats(N, B, fmt, **more):
    return {"op": "stats", "N": N, "B": B, "fmt": fmt, **more}


def _apply(N, B, fmt, diag=True, **more):
    return {"op": "apply", "N": N, "B": B, "fmt": fmt, "diag": diag, **more}


def _grad(T, out, inp, B, type, fmt="e4m3", accumulate=False, **more):
    return {"op": "grad", "T": T, "out": out, "in": inp, "B": B, "type": type, "fmt": fmt, "accumulate": accumulate,
            **more}


def listed():
    return [
        # the smallest stack, where a call is its launch: four 64-wide roots to 4 bits
        _quantize(4, 64, 64, "fp32", "e2m1", "rows", True, name="roots_4x64_e2m1"),
        # a layer's input saved in the forward pass: 8 sequences of 1024 tokens, embedding 2048
        _quantize(1, 8192, 2048, "bf16", "e4m3", "rows", name="acts_8192x2048_e4m3"),
        # an odd activation: neither side a multiple of a group, rows of no particular alignment
        _quantize(1, 1777, 1001, "fp16", "e4m3", "both", name="acts_1777x1001_both"),
        # gradient tiles for both statistics: rows for G G^T, columns for G^T G
        _quantize(192, 1024, 1024, "fp32", "e4m3", "both", name="tiles_192x1024_both"),
        # statistics of a small model's tiles
        _stats(8, 192, "e2m1", name="stats_8x192_e2m1"),
        # statistics of 384 tiles of 1024 (six layers of the benchmark's model)
        _stats(384, 1024, "e4m3", name="stats_384x1024_e4m3"),
        # the update of one small weight's tiles
        _apply(2, 128, "e2m1", name="apply_2x128_e2m1"),
        # the update of the same 384 tiles, roots kept in 4 bits
        _apply(384, 1024, "e2m1", name="apply_384x1024_e2m1"),
        # one token's contribution to a small layer
        _grad(1, 256, 192, 64, "bf16", name="grad_1x256x192"),
        # a long batch of a narrow layer, added to the earlier micro-batches' sum: few tiles, many tokens
        _grad(50000, 520, 264, 256, "fp32", accumulate=True, name="grad_50000x520x264_fp32"),
        # an attention projection of the benchmark's model, one micro-batch
        _grad(4096, 2048, 2048, 1024, "bf16", name="grad_4096x2048x2048"),
        # an MLP weight of the benchmark's model, a whole batch
        _grad(16384, 2048, 8192, 1024, "bf16", name="grad_16384x2048x8192"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "stats", "apply", "grad"))
    fmt = rng.choice(FMTS)
    if op == "quantize":
        type = rng.choice(tuple(TYPES))
        if rng.random() < 0.5:  # a stack of tiles or roots
            B = 64 * _log(rng, 1, 32)
            N = _log(rng, 1, max(1, 192 * 1024 * 1024 // (B * B)))
            return _quantize(N, B, B, "fp32", fmt, rng.choice(("rows", "cols", "both")), rng.random() < 0.5)
        return _quantize(1, _log(rng, 1, 16384), _log(rng, 1, 8192), type, fmt, rng.choice(("rows", "cols", "both")))
    if op in ("stats", "apply"):
        B = 64 * _log(rng, 1, 32)
        N = _log(rng, 1, max(1, min(20000, 384 * 1024**3 // B**3 // 2, 384 * 1024 * 1024 // (B * B))))
        return _stats(N, B, fmt) if op == "stats" else _apply(N, B, fmt, rng.random() < 0.7)
    out, inp = _log(rng, 1, 8192), _log(rng, 1, 8192)
    T = _log(rng, 1, max(1, min(65536, 2**37 // (out * inp))))
    B = 64 * _log(rng, 1, 32)
    return _grad(T, out, inp, B, rng.choice(tuple(TYPES)), fmt, rng.random() < 0.3)


def work(case):
    """What one pass cannot do without: each input read once, each output written once."""
    c, g = case, lambda n: -(-n // GROUP)
    width = {"e2m1": 0.5, "e4m3": 1.0}[c["fmt"]]
    size = {"fp32": 4, "bf16": 2, "fp16": 2}.get(c.get("type"), 4)
    if c["op"] == "quantize":
        n = c["N"] * c["rows"] * c["cols"]
        sides = 2 if c["sides"] == "both" else 1
        back = 4 if c["type"] == "fp32" else 2
        # codes and scales written and read back, the values that they stand for written
        return {"bytes": n * (size + sides * (2 * (width + 1 / GROUP) + back)), "flops": n * sides * 2.0}
    if c["op"] == "stats":
        n = c["N"] * c["B"] ** 2
        return {"bytes": n * (2 * (width + 1 / GROUP) + 2 * 2 + 2 * 4), "flops": 2.0 * n * (c["B"] + 1)}
    if c["op"] == "apply":
        n = c["N"] * c["B"] ** 2
        return {"bytes": n * (2 * (width + 1 / GROUP) + 4 + 4), "flops": 4.0 * n * c["B"]}
    tiles = -(-c["out"] // c["B"]) * -(-c["in"] // c["B"]) * c["B"] ** 2
    rw = 2 if c["accumulate"] else 1
    return {"bytes": c["T"] * (c["out"] * size + c["in"] * (width + 1 / GROUP)) + 4 * tiles * rw,
            "flops": 2.0 * c["T"] * c["out"] * c["in"]}


# ------------------------------------------------------------------------------------------------
# The plain form
# ------------------------------------------------------------------------------------------------


def _groups(x):
    """The last axis in groups of 32, the last of them padded with zeros."""
    pad = -x.shape[-1] % GROUP
    x = torch.nn.functional.pad(x, (0, pad)) if pad else x
    return x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)


def _plain_quantize(x, fmt):
    """(codes, scale bytes, values) of the rows of x [..., cols], in 32 bits."""
    cols = x.shape[-1]
    v = _groups(x.float())
    top = v.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(top)
    frac, expo = torch.frexp(torch.where(bad, torch.ones_like(top), top))
    # m = 0.75 2^3 or 0.875 2^9: the least e with top <= m 2^e
    half, at = (0.75, 3) if fmt == "e2m1" else (0.875, 9)
    e = expo - at + (frac > half).int()
    e = torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    y = torch.where(bad, torch.zeros_like(v), torch.ldexp(torch.ldexp(v, -(e // 2)), -(e - e // 2)))
    a = y.abs()
    _, ye = torch.frexp(a)
    lowest, bits = (0, 1) if fmt == "e2m1" else (-6, 3)
    ulp = (ye - 1).clamp(min=lowest) - bits  # exponent of the grid's step at a
    q = torch.round(torch.ldexp(a, -ulp))  # a whole number of steps, ties to even
    r = torch.ldexp(q, ulp)  # |element|, on the grid
    _, re = torch.frexp(r)
    re = torch.where(r > 0, re - 1, torch.full_like(re, lowest)).clamp(min=lowest)
    steps = torch.ldexp(r, bits - re).int()  # 2^bits + mantissa, or the mantissa of a subnormal
    code = torch.where(steps >= 2**bits, (re - lowest + 1) * 2**bits + steps - 2**bits, steps)
    code = code + (torch.signbit(y).int() << (3 if fmt == "e2m1" else 7))
    scale = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    code = code.to(torch.uint8)
    codes = code.reshape(*x.shape[:-1], -1)
    if fmt == "e2m1":
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes.contiguous(), scale.reshape(*x.shape[:-1], -1).contiguous()


def _plain_values(codes, scales, cols, fmt):
    """The values that codes and scale bytes stand for, in 32 bits."""
    if fmt == "e2m1":
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).int()
        v = table[c & 7]
        v = torch.where(c > 7, -v, v)
    else:
        c = codes.int()
        ex, ma = (c >> 3) & 15, (c & 7).float()
        v = torch.where(ex > 0, torch.ldexp(8 + ma, ex - 10), ma / 512)
        v = torch.where(c > 127, -v, v)
    e = scales.int() - 127
    half = torch.div(e, 2, rounding_mode="floor")
    v = v.reshape(*v.shape[:-1], -1, GROUP)
    v = torch.ldexp(torch.ldexp(v, half[..., None]), (e - half)[..., None])
    v = torch.where((scales == 255)[..., None], torch.full_like(v, float("nan")), v)
    return v.reshape(*codes.shape[:-1], -1)[..., :cols]


def _tiles(W, B):
    """The B x B tiles of W, row by row, edge tiles padded with zeros."""
    r, c = -(-W.shape[0] // B), -(-W.shape[1] // B)
    W = torch.nn.functional.pad(W, (0, c * B - W.shape[1], 0, r * B - W.shape[0]))
    return W.reshape(r, B, c, B).permute(0, 2, 1, 3).reshape(r * c, B, B)


def _plain(c, s):
    fmt = c["fmt"]
    if c["op"] == "quantize":
        x, out = s["x"], {}
        if c["diag"]:
            d = torch.diagonal(x, dim1=1, dim2=2)
            x = x - torch.diag_embed(d)
            out["diag"] = d.float().contiguous()
        back = torch.float32 if c["type"] == "fp32" else torch.bfloat16
        for side in ("rows", "cols"):
            if c["sides"] in (side, "both"):
                y = x if side == "rows" else x.transpose(1, 2)
                codes, scales = _plain_quantize(y, fmt)
                v = _plain_values(codes, scales, y.shape[-1], fmt)
                if c["diag"]:
                    v = v + torch.diag_embed(out["diag"])
                out[side], out[side + "_scales"] = v.to(back), scales
        return out
    if c["op"] == "stats":
        A, N, B = s["A"], c["N"], c["B"]
        g = _plain_values(s["codes"], s["scales"], B, fmt)
        A[:N].mul_(s["beta"]).add_(torch.matmul(g, g.transpose(1, 2).contiguous()), alpha=1 - s["beta"])
        g = _plain_values(s["codes_t"], s["scales_t"], B, fmt)
        A[N:].mul_(s["beta"]).add_(torch.matmul(g, g.transpose(1, 2).contiguous()), alpha=1 - s["beta"])
        return A
    if c["op"] == "apply":
        L = _plain_values(s["XL"], s["XL_scales"], c["B"], fmt)
        R = _plain_values(s["XR"], s["XR_scales"], c["B"], fmt)
        if c["diag"]:
            L, R = L + torch.diag_embed(s["XL_diag"]), R + torch.diag_embed(s["XR_diag"])
        return torch.matmul(torch.matmul(L, s["G"]), R.transpose(1, 2).contiguous())
    X = _plain_values(s["codes"], s["scales"], c["in"], fmt)
    tiles = _tiles(torch.matmul(s["dY"].float().t().contiguous(), X), c["B"])
    if c["accumulate"]:
        return s["G"].add_(tiles)
    return s["G"].copy_(tiles)


# ------------------------------------------------------------------------------------------------
# The library's calls
# ------------------------------------------------------------------------------------------------


def _own(c, s):
    import matrix_inverse_roots_amd as dash

    fmt = {"e2m1": dash.DASH_MX_E2M1, "e4m3": dash.DASH_MX_E4M3}[c["fmt"]]
    if c["op"] == "quantize":
        N, rows, cols = s["x"].shape
        back = torch.float32 if c["type"] == "fp32" else torch.bfloat16
        pair, out = {}, {}
        for side, shape in (("rows", (N, rows, cols)), ("cols", (N, cols, rows))):
            pair[side] = dash.mx_buffers(*shape, fmt, device=DEV) if c["sides"] in (side, "both") else (None, None)
        diag = torch.empty((N, rows), device=DEV) if c["diag"] else None
        dash.dash_mx_quantize(s["x"], N, rows, cols, fmt, *pair["rows"], *pair["cols"], diag=diag)
        for side, shape in (("rows", (N, rows, cols)), ("cols", (N, cols, rows))):
            codes, scales = pair[side]
            if codes is not None:
                v = torch.empty(shape, dtype=back, device=DEV)
                dash.dash_mx_dequantize(codes, scales, *shape, fmt, v, diag=diag)
                out[side], out[side + "_scales"] = v, scales
        if diag is not None:
            out["diag"] = diag
        return out
    if c["op"] == "stats":
        dash.dash_update_stats_mx(s["codes"], s["scales"], s["codes_t"], s["scales_t"], c["N"], c["B"], fmt, s["beta"],
                                  s["A"])
        return s["A"]
    if c["op"] == "apply":
        if "ws" not in s:
            s["ws"] = dash.workspace(dash.DASH_OP_APPLY, c["N"], c["B"], device=DEV)
            s["U"] = torch.empty_like(s["G"])
        dash.dash_apply_mx(s["XL"], s["XL_scales"], s["XR"], s["XR_scales"], s["G"], c["N"], c["B"], fmt, s["U"],
                           XL_diag=s.get("XL_diag"), XR_diag=s.get("XR_diag"), ws=s["ws"])
        return s["U"]
    if "ws" not in s:
        s["ws"] = dash.grad_stack_mx_workspace(c["T"], c["out"], c["in"], s["dY"].dtype, device=DEV)
        s["G"] = s["G"].contiguous()  # (one row of tiles may have come as a strided view)
    dash.dash_grad_stack_mx(s["dY"], s["codes"], s["scales"], fmt, c["T"], c["out"], c["in"], c["B"], s["G"],
                            accumulate=c["accumulate"], ws=s["ws"])
    return s["G"]


# ------------------------------------------------------------------------------------------------
# Inputs, a pass, and the definition in 64 bits
# ------------------------------------------------------------------------------------------------


def _roots(gen, N, B):
    """Inverse fourth roots as a run meets them: symmetric, their diagonals well above the rest, each
    block of its own magnitude."""
    S = torch.randn((N, B, B), generator=gen, device=DEV)
    X = (S + S.transpose(1, 2)) * (0.1 / math.sqrt(B))
    d = 1 + 0.5 * torch.rand((N, B), generator=gen, device=DEV)
    size = torch.pow(10.0, 2 * torch.rand((N, 1, 1), generator=gen, device=DEV))
    return (X + torch.diag_embed(d)) * size


def _activations(gen, T, n):
    """A layer's input: tokens of unequal size, and a few channels far above the others."""
    x = torch.randn((T, n), generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=gen, device=DEV))
    x *= torch.where(torch.rand(n, generator=gen, device=DEV) < 0.01, 30.0, 1.0)
    return x


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "quantize":
        if c["diag"]:
            s["x"] = _roots(gen, c["N"], c["rows"])
        elif c["N"] > 1:  # gradient tiles
            s["x"] = 1e-3 * torch.randn((c["N"], c["rows"], c["cols"]), generator=gen, device=DEV)
        else:
            s["x"] = _activations(gen, c["rows"], c["cols"])[None].to(TYPES[c["type"]])
    elif c["op"] == "stats":
        N, B = c["N"], c["B"]
        G = 1e-3 * torch.randn((N, B, B), generator=gen, device=DEV)
        s["codes"], s["scales"] = _plain_quantize(G, c["fmt"])
        s["codes_t"], s["scales_t"] = _plain_quantize(G.transpose(1, 2), c["fmt"])
        S = torch.randn((2 * N, B, B), generator=gen, device=DEV)
        s["A"] = (S + S.transpose(1, 2)) * 1e-6
        s["beta"] = 0.95
    elif c["op"] == "apply":
        N, B = c["N"], c["B"]
        for side in ("XL", "XR"):
            X = _roots(gen, N, B)
            if c["diag"]:
                s[side + "_diag"] = torch.diagonal(X, dim1=1, dim2=2).contiguous()
                X = X - torch.diag_embed(s[side + "_diag"])
            s[side], s[side + "_scales"] = _plain_quantize(X, c["fmt"])
        s["G"] = 1e-3 * torch.randn((N, B, B), generator=gen, device=DEV)
    else:
        s["codes"], s["scales"] = _plain_quantize(_activations(gen, c["T"], c["in"]), c["fmt"])
        s["dY"] = (1e-3 * torch.randn((c["T"], -(-c["out"] // 8) * 8), generator=gen, device=DEV)).to(TYPES[c["type"]])
        s["dY"] = s["dY"][:, : c["out"]]
        shape = (-(-c["out"] // c["B"]) * -(-c["in"] // c["B"]), c["B"], c["B"])
        # the earlier micro-batches' sum, whose padding is zero
        G = 1e-3 * torch.randn((c["out"], c["in"]), generator=gen, device=DEV) if c["accumulate"] else None
        s["G"] = torch.empty(shape, device=DEV) if G is None else _tiles(G, c["B"])
    return s


def run(state):
    return _own(state["case"], state) if own else _plain(state["case"], state)


def _exact_grid(fmt):
    """Every non-negative element value in ascending order (its place is its code)."""
    if fmt == "e2m1":
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    low = [m * 2.0**-9 for m in range(8)]
    high = [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor((low + high)[:127], dtype=torch.float64, device=DEV)  # the last one is no number


def _exact_rows(x, fmt):
    """(values, scale bytes) of x [rows, cols] in 64 bits: the nearest grid value by search."""
    rows, cols = x.shape
    n = -(-cols // GROUP)
    v = torch.zeros((rows, n * GROUP), dtype=torch.float64, device=DEV)
    v[:, :cols] = x.double()
    v = v.view(rows, n, GROUP)
    top = v.abs().max(dim=2).values
    e = torch.ceil(torch.log2(top / TOP[fmt])).clamp(-127, 127)
    e = e - (top <= TOP[fmt] * torch.exp2(e - 1)).double()  # (the logarithm may be off at a border)
    e = (e + (top > TOP[fmt] * torch.exp2(e)).double()).clamp(-127, 127)
    grid = _exact_grid(fmt)
    step = torch.exp2(e)[:, :, None]
    a = (v.abs() / step).clamp(max=TOP[fmt])
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    q = grid[pick] * torch.sign(v) * step
    return q.view(rows, n * GROUP)[:, :cols], (e + 127).to(torch.uint8)


def _exact_values(codes, scales, cols, fmt):
    grid = _exact_grid(fmt)
    if fmt == "e2m1":
        signed = torch.cat((grid, -grid))
        v = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device=DEV)
        v[..., 0::2], v[..., 1::2] = signed[(codes % 16).long()], signed[(codes // 16).long()]
    else:
        last = torch.full((1,), float("nan"), dtype=torch.float64, device=DEV)
        v = torch.cat((grid, last, -grid, last))[codes.long()]
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(GROUP, -1))[..., :cols]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    fmt = c["fmt"]
    if c["op"] == "quantize":
        N, rows, cols = s["x"].shape
        out = {}
        x = s["x"].double()
        keep = 0.0
        if c["diag"]:
            eye = torch.eye(rows, dtype=torch.float64, device=DEV)
            keep = x * eye
            x = x - keep
            out["diag"] = keep.sum(2)
        for side, m in (("rows", x), ("cols", x.permute(0, 2, 1))):
            if c["sides"] in (side, "both"):
                flat = m.reshape(-1, m.shape[2])
                at = [_exact_rows(b, fmt) for b in flat.split(max(1, 2**25 // m.shape[2]))]
                out[side] = torch.cat([q for q, _ in at]).view(m.shape) + keep
                out[side + "_scales"] = torch.cat([q for _, q in at]).view(N, m.shape[1], -1)
        return out
    if c["op"] == "stats":
        N, B = c["N"], c["B"]
        new = torch.empty((2 * N, B, B), dtype=torch.float64, device=DEV)
        for i in range(2 * N):
            side = "" if i < N else "_t"
            g = _exact_values(s["codes" + side][i % N], s["scales" + side][i % N], B, fmt)
            new[i] = s["A"][i].double() * s["beta"] + (1 - s["beta"]) * (g @ g.T)
        return new
    if c["op"] == "apply":
        N, B = c["N"], c["B"]
        U = torch.empty((N, B, B), dtype=torch.float64, device=DEV)
        for i in range(N):
            X = []
            for side in ("XL", "XR"):
                X.append(_exact_values(s[side][i], s[side + "_scales"][i], B, fmt))
                if c["diag"]:
                    X[-1] += torch.diag(s[side + "_diag"][i].double())
            U[i] = X[0] @ s["G"][i].double() @ X[1].T
        return U
    T, out, inp, B = c["T"], c["out"], c["in"], c["B"]
    W = torch.zeros((out, inp), dtype=torch.float64, device=DEV)
    for t in range(0, T, 4096):
        x = _exact_values(s["codes"][t : t + 4096], s["scales"][t : t + 4096], inp, fmt)
        W += s["dY"][t : t + 4096].double().T @ x
    nr, nc = -(-out // B), -(-inp // B)
    G = torch.zeros((nr * nc, B, B), dtype=torch.float64, device=DEV)
    for i in range(nr * nc):
        part = W[i // nc * B : (i // nc + 1) * B, i % nc * B : (i % nc + 1) * B]
        G[i, : part.shape[0], : part.shape[1]] = part
    return G + s["G"].double() if c["accumulate"] else G
