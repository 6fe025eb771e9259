"""Cases and plain forms of the operators between a layer's norm and the statistics: the
root-mean-square norm with the residual's addition and a microscaled output, its gradient, the global
norm of many gradients, and clipping (in place, or on the way into gradient tiles).

  norm      h = x + res, rstd = (mean h^2 + eps)^-1/2, y = h rstd gain; y also as microscaled rows
            (groups of 32 along a row, the last padded with zeros, E4M3 elements and one power of two each:
            2^e with the least e >= -127 that keeps the group's largest magnitude within 448 2^e)
  gradient  m = dy gain, xhat = h rstd: dx = dh + rstd (m - xhat mean(m xhat)), dgain += sum_t dy xhat
  grads     |g_i| of every tensor and the square root of the sum of their squares
  clip      g min(1, most / norm), in place, or as B x B tiles of the weights

`run` computes the plain form (elementary torch operations in 32 bits, long sums in 64) unless `own` is
set, and calls the library then.  `exact` is the same in 64 bits, written from the definitions.  Codes and
scale bytes are returned as the numbers they hold: E4M3 elements, and powers of two.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-5


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------


def _norm(T, n, type, res=True, y=True, gain="fp32", **more):
    return {"op": "norm", "T": T, "n": n, "type": type, "res": res, "y": y, "gain": gain, **more}


def _back(T, n, type, dh=True, accumulate=False, gain="fp32", **more):
    return {"op": "back", "T": T, "n": n, "type": type, "dh": dh, "accumulate": accumulate, "gain": gain, **more}


def _grads(layers=0, count=0, most=0, shapes=0, type="fp32", **more):
    """`layers` of the benchmark's model (and its norms' gains), or `count` tensors of up to `most` elements."""
    return {"op": "grads", "layers": layers, "count": count, "most": most, "shapes": shapes, "type": type, **more}


def _clip(into, layers=0, count=0, most=0, shapes=0, type="fp32", B=1024, **more):
    return {"op": "clip", "into": into, "layers": layers, "count": count, "most": most, "shapes": shapes,
            "type": type, "B": B, **more}


def listed():
    return [
        # one token of a sequence that is being continued: the call is its launch
        _norm(1, 2048, "bf16", gain="bf16", name="norm_1x2048_bf16"),
        # rows of an odd length, on no alignment; only the 8-bit checkpoint is kept, no residual
        _norm(1777, 1001, "fp16", res=False, y=False, gain="fp16", name="norm_1777x1001_fp16"),
        # a training step's norm: 8 sequences of 1024 tokens, embedding 2048
        _norm(8192, 2048, "bf16", gain="bf16", name="norm_8192x2048_bf16"),
        # a long batch at the MLP's width, the residual stream in 32 bits
        _norm(32768, 8192, "fp32", y=False, name="norm_32768x8192_fp32"),
        # the gradient of a few tokens
        _back(16, 2048, "bf16", gain="bf16", name="back_16x2048_bf16"),
        # many tokens, narrow rows of an odd length: the sum over tokens is what is long; a later micro-batch
        _back(50001, 263, "fp32", accumulate=True, name="back_50001x263_fp32"),
        # the gradient of a long batch at the MLP's width
        _back(32768, 8192, "bf16", gain="bf16", name="back_32768x8192_bf16"),
        # the biases and gains of one layer
        _grads(count=9, most=2048, shapes=1, type="mixed", name="grads_9_small"),
        # every gradient of the benchmark's model: 24 layers of 7 weights and 2 gains
        _grads(layers=24, name="grads_model"),
        # a model of many odd tensors in place: pieces of larger buffers, three types, any alignment
        _clip("place", count=1000, most=1 << 20, shapes=2, type="mixed", name="clip_1000_ragged"),
        # six layers in 16 bits in place
        _clip("place", layers=6, type="bf16", name="clip_six_layers_bf16"),
        # norm, then clipped into the tiles that the statistics take: six layers, 384 tiles of 1024
        _clip("tiles", layers=6, name="tiles_six_layers"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "back", "back", "grads", "clip", "clip"))
    if op in ("norm", "back"):
        n = _log(rng, 8, 16384)  # (in a row of one or two, the terms of dx cancel but for their rounding)
        T = _log(rng, 1, max(1, min(65536, 2**28 // n)))
        type = rng.choice(tuple(TYPES))
        gain = rng.choice((type, "fp32"))
        if op == "norm":
            return _norm(T, n, type, rng.random() < 0.7, rng.random() < 0.7, gain)
        return _back(T, n, type, rng.random() < 0.7, rng.random() < 0.3, gain)
    into = rng.choice(("place", "tiles")) if op == "clip" else None
    type = "fp32" if into == "tiles" else rng.choice(tuple(TYPES) + ("mixed",))
    B = 64 * _log(rng, 1, 32)
    if rng.random() < 0.3:
        size = {"layers": _log(rng, 1, 6)}
    else:
        count = _log(rng, 1, 1000)
        size = {"count": count, "most": _log(rng, 16, max(16, 2**29 // count)), "shapes": rng.randrange(1 << 16)}
    if op == "grads":
        return _grads(type=type, **size)
    case = _clip(into, type=type, B=B, **size)
    while into == "tiles" and _tile_count(case) * case["B"] ** 2 > 2**29:  # (a tile may hold a single element)
        if case["B"] > 64:
            case["B"] = max(64, case["B"] // 2 // 64 * 64)
        else:
            case["most"] //= 2
    return case


def _shapes(c):
    """(rows, columns, row pitch, type) of every tensor of a case; a vector has one row."""
    one = c["type"] if c["type"] != "mixed" else "fp32"
    if c["layers"]:
        d, ffn = 2048, 8192
        layer = [(d, d)] * 4 + [(ffn, d)] * 2 + [(d, ffn)]
        if c.get("into") != "tiles":  # (gains are vectors: they have no tiles)
            layer = layer + [(1, d)] * 2
        return [(r, k, k, one) for r, k in layer * c["layers"]]
    rng = random.Random(c["shapes"])
    out = []
    for _ in range(c["count"]):
        size = _log(rng, 1, c["most"])
        type = rng.choice(tuple(TYPES)) if c["type"] == "mixed" else one
        if c.get("into") == "tiles":  # rows that start on 16 bytes, as stacking takes them
            r = _log(rng, 1, size)
            k = max(1, size // r)
            out.append((r, k, k + -k % 4 + 4 * rng.randrange(3), type))
        elif rng.random() < 0.3:  # a slice of a wider matrix
            r = _log(rng, 1, size)
            k = max(1, size // r)
            out.append((r, k, k + rng.randrange(1, 9), type))
        else:
            out.append((1, size, size, type))
    return out


def _tile_count(c):
    return sum(-(-r // c["B"]) * -(-k // c["B"]) for r, k, _, _ in _shapes(c))


def work(case):
    """What one pass cannot do without: each input read once, each output written once."""
    c = case
    if c["op"] in ("norm", "back"):
        size = {"fp32": 4, "bf16": 2, "fp16": 2}
        s, T, n = size[c["type"]], c["T"], c["n"]
        if c["op"] == "norm":
            streams = 1 + 2 * c["res"] + c["y"]  # x; the residual and its new state; y
            return {"bytes": T * (n * s * streams + -(-n // GROUP) * (GROUP + 1) + 4) + n * size[c["gain"]],
                    "flops": 6.0 * T * n}
        return {"bytes": T * (n * s * (3 + c["dh"]) + 4) + n * (size[c["gain"]] + 4 * (1 + c["accumulate"])),
                "flops": 10.0 * T * n}
    read = sum(r * k * (4 if t == "fp32" else 2) for r, k, _, t in _shapes(c))
    n = sum(r * k for r, k, _, _ in _shapes(c))
    if c["op"] == "grads":
        return {"bytes": read + 4 * len(_shapes(c)), "flops": 2.0 * n}
    if c["into"] == "place":
        return {"bytes": 2 * read, "flops": 1.0 * n}
    return {"bytes": read + 4 * _tile_count(c) * c["B"] ** 2, "flops": 3.0 * n}


# ------------------------------------------------------------------------------------------------
# The plain form
# ------------------------------------------------------------------------------------------------


def _plain_rows(y):
    """(elements, scales) of the microscaled rows of y [T, n], in 32 bits."""
    T, n = y.shape
    v = torch.nn.functional.pad(y, (0, -n % GROUP)).reshape(T, -1, GROUP)
    top = v.abs().amax(-1, keepdim=True)
    frac, expo = torch.frexp(top)
    e = expo - 9 + (frac > 0.875).int()  # 448 = 0.875 2^9
    e = torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    q = torch.ldexp(torch.ldexp(v, -(e // 2)), -(e - e // 2)).to(torch.float8_e4m3fn)
    byte = (e + 127).to(torch.uint8)
    return q.reshape(T, -1), byte.reshape(T, -1).view(torch.float8_e8m0fnu)


def _tiles(W, B):
    """The B x B tiles of W, row by row, edge tiles padded with zeros."""
    r, c = -(-W.shape[0] // B), -(-W.shape[1] // B)
    W = torch.nn.functional.pad(W, (0, c * B - W.shape[1], 0, r * B - W.shape[0]))
    return W.reshape(r, B, c, B).permute(0, 2, 1, 3).reshape(r * c, B, B)


def _plain_norms(grads):
    sums = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads])
    return sums.sum().sqrt().float().reshape(1), sums.sqrt().float()


def _plain(c, s):
    if c["op"] == "norm":
        h = s["x"].float()
        if c["res"]:
            h = h + s["res"].float()
        rstd = torch.rsqrt(h.square().mean(-1) + EPS)
        y = h * rstd[:, None] * s["gain"].float()
        out = {"rstd": rstd}
        out["codes"], out["scales"] = _plain_rows(y)
        if c["res"]:
            out["h"] = h.to(s["x"].dtype)
        if c["y"]:
            out["y"] = y.to(s["x"].dtype)
        return out
    if c["op"] == "back":
        dy, xhat = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        m = dy * s["gain"].float()
        dx = (m - xhat * (m * xhat).mean(-1, keepdim=True)) * s["rstd"][:, None]
        if c["dh"]:
            dx = dx + s["dh"].float()
        dgain = (dy * xhat).sum(0)
        s["dgain"] = s["dgain"].add_(dgain) if c["accumulate"] else s["dgain"].copy_(dgain)
        return {"dx": dx.to(s["dy"].dtype), "dgain": s["dgain"]}
    if c["op"] == "grads":
        norm, norms = _plain_norms(s["grads"])
        return {"norm": norm, "norms": norms}
    if c["into"] == "tiles":
        norm, _ = _plain_norms(s["grads"])
        factor = (s["most"] / norm).clamp(max=1.0)
        return {"norm": norm, "tiles": torch.cat([_tiles(g * factor, c["B"]) for g in s["grads"]])}
    factor = (s["most"] / s["norm"]).clamp(max=1.0)
    for g in s["grads"]:
        g.copy_(g.float() * factor)
    return s["flat"]


# ------------------------------------------------------------------------------------------------
# The library's calls
# ------------------------------------------------------------------------------------------------


def _own(c, s):
    import matrix_inverse_roots_amd as dash

    if c["op"] == "norm":
        T, n = s["x"].shape
        if "codes" not in s:  # buffers that a training program keeps from step to step
            s["codes"], s["scales"] = dash.mx_buffers(1, T, n, dash.DASH_MX_E4M3, device=DEV)
            s["rstd"] = torch.empty(T, device=DEV)
            s["h"] = torch.empty_like(s["x"]) if c["res"] else None
            s["y"] = torch.empty_like(s["x"]) if c["y"] else None
        dash.dash_rmsnorm(s["x"], T, n, EPS, res=s["res"], gain=s["gain"], h=s["h"], y=s["y"],
                          fmt=dash.DASH_MX_E4M3, codes=s["codes"], scales=s["scales"], rstd=s["rstd"])
        out = {"rstd": s["rstd"], "codes": s["codes"][0].view(torch.float8_e4m3fn),
               "scales": s["scales"][0].view(torch.float8_e8m0fnu)}
        if c["res"]:
            out["h"] = s["h"]
        if c["y"]:
            out["y"] = s["y"]
        return out
    if c["op"] == "back":
        T, n = s["dy"].shape
        if "ws" not in s:
            s["ws"] = dash.rmsnorm_backward_workspace(T, n, device=DEV)
            s["dx"] = torch.empty_like(s["dy"])
        dash.dash_rmsnorm_backward(s["dy"], s["h"], s["rstd"], T, n, s["dx"], gain=s["gain"], dh=s["dh"],
                                   dgain=s["dgain"], accumulate=c["accumulate"], ws=s["ws"])
        return {"dx": s["dx"], "dgain": s["dgain"]}
    if "list" not in s:  # the gradients' buffers stay, and so does what describes them
        s["list"] = dash.grad_list(s["grads"])
        s["ws"] = dash.grad_norm_workspace(s["list"], device=DEV)
    if c["op"] == "grads":
        if "norm" not in s:
            s["norm"], s["norms"] = torch.empty(1, device=DEV), torch.empty(len(s["grads"]), device=DEV)
        dash.dash_grad_norm(s["list"], s["norm"], norms=s["norms"], ws=s["ws"])
        return {"norm": s["norm"], "norms": s["norms"]}
    if c["into"] == "tiles":
        if "tiles" not in s:
            s["norm"] = torch.empty(1, device=DEV)
            s["tiles"] = torch.empty((_tile_count(c), c["B"], c["B"]), device=DEV)
        dash.dash_grad_norm(s["list"], s["norm"], ws=s["ws"])
        dash.dash_stack_clip(s["list"], c["B"], s["norm"], s["most"], s["tiles"])
        return {"norm": s["norm"], "tiles": s["tiles"]}
    dash.dash_grad_clip(s["list"], s["norm"], s["most"])
    return s["flat"]


# ------------------------------------------------------------------------------------------------
# Inputs, a pass, and the definition in 64 bits
# ------------------------------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _activations(gen, T, n):
    """A residual stream: tokens of unequal size, and a few channels far above the others."""
    x = _randn(gen, T, n)
    x *= torch.exp(0.5 * _randn(gen, T, 1))
    return x.mul_(torch.where(torch.rand(n, generator=gen, device=DEV) < 0.01, 30.0, 1.0))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("norm", "back"):
        T, n, type = c["T"], c["n"], TYPES[c["type"]]
        s["gain"] = (1 + 0.2 * _randn(gen, n)).to(TYPES[c["gain"]])
        x = _activations(gen, T, n).to(type)
        if c["op"] == "norm":
            s["x"], s["res"] = x, None
            if c["res"]:  # x is a layer's output, a part of the stream that it is added to
                s["res"] = _activations(gen, T, n).mul_(2).to(type)
            return s
        s["h"] = x
        s["rstd"] = torch.rsqrt(x.float().square().mean(-1) + EPS)
        s["dy"] = (1e-3 * _randn(gen, T, n)).to(type)
        s["dh"] = (1e-3 * _randn(gen, T, n)).to(type) if c["dh"] else None
        s["dgain"] = 1e-2 * _randn(gen, n) if c["accumulate"] else torch.empty(n, device=DEV)
        return s
    shapes = _shapes(c)
    place, at = [], {t: 0 for t in TYPES}
    rng = random.Random(c["shapes"])
    for r, k, ld, t in shapes:  # in buffers of one type each, one after the other
        if c["layers"] or c.get("into") == "tiles":
            at[t] += -at[t] % 8
        else:
            at[t] += rng.randrange(8)
        place.append(at[t])
        at[t] += r * ld
    s["flat"] = {t: (1e-3 * _randn(gen, size)).to(TYPES[t]) for t, size in at.items() if size}
    s["grads"] = [s["flat"][t][p:p + k] if r == 1 else s["flat"][t].as_strided((r, k), (ld, 1), p)
                  for p, (r, k, ld, t) in zip(place, shapes)]
    if c.get("into") == "tiles":
        s["grads"] = [g if g.dim() == 2 else g[None] for g in s["grads"]]
        # (one row keeps its pitch)
        s["grads"] = [g.as_strided(g.shape, (sh[2], 1)) for g, sh in zip(s["grads"], shapes)]
    if c["op"] == "clip":
        count = sum(r * k for r, k, _, _ in shapes)
        s["most"] = 1e-3 * math.sqrt(count) * (0.3 + 0.5 * random.Random(seed).random())
        if c["into"] == "place":  # the norm over all ranks, from the step that reduced it
            s["norm"] = torch.full((1,), 1e-3 * math.sqrt(count), device=DEV)
    return s


def run(state):
    return _own(state["case"], state) if own else _plain(state["case"], state)


def _exact_rows(y):
    """(element values, powers of two) of the rows of y [T, n] in 64 bits: the nearest element by search."""
    T, n = y.shape
    g = -(-n // GROUP)
    v = torch.zeros((T, g * GROUP), dtype=torch.float64, device=DEV)
    v[:, :n] = y
    v = v.view(T, g, GROUP)
    top = v.abs().max(dim=2).values
    e = torch.ceil(torch.log2(top / 448)).clamp(-127, 127)
    e = e - (top <= 448 * torch.exp2(e - 1)).double()  # (the logarithm may be off at a border)
    e = (e + (top > 448 * torch.exp2(e)).double()).clamp(-127, 127)
    low = [m * 2.0**-9 for m in range(8)]
    high = [(1 + m / 8) * 2.0 ** (k - 7) for k in range(1, 16) for m in range(8)]
    grid = torch.tensor((low + high)[:127], dtype=torch.float64, device=DEV)
    a = (v.abs() / torch.exp2(e)[:, :, None]).clamp(max=448.0)
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (grid[pick] * torch.sign(v)).view(T, -1), torch.exp2(e)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        T, n = s["x"].shape
        parts = []
        for t in range(0, T, max(1, 2**25 // n)):
            rows = slice(t, t + max(1, 2**25 // n))
            h = s["x"][rows].double()
            if c["res"]:
                h += s["res"][rows].double()
            rstd = 1 / torch.sqrt((h * h).sum(1) / n + EPS)
            y = h * rstd[:, None] * s["gain"].double()
            q, e = _exact_rows(y)
            part = {"rstd": rstd, "codes": q, "scales": e}
            if c["res"]:
                part["h"] = h
            if c["y"]:
                part["y"] = y
            parts.append(part)
        return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if c["op"] == "back":
        T, n = s["dy"].shape
        dgain = s["dgain"].double() if c["accumulate"] else torch.zeros(n, dtype=torch.float64, device=DEV)
        dx = torch.empty((T, n), dtype=torch.float64, device=DEV)
        gain = s["gain"].double()
        for t in range(0, T, max(1, 2**25 // n)):
            rows = slice(t, t + max(1, 2**25 // n))
            r = s["rstd"][rows].double()[:, None]
            dy, h = s["dy"][rows].double(), s["h"][rows].double()
            dgain += (dy * h * r).sum(0)
            dot = (dy * gain * h).sum(1, keepdim=True)
            dx[rows] = r * dy * gain - r**3 * h * dot / n
            if c["dh"]:
                dx[rows] += s["dh"][rows].double()
        return {"dx": dx, "dgain": dgain}
    norms = torch.tensor([float(torch.linalg.vector_norm(g.double())) for g in s["grads"]], dtype=torch.float64,
                         device=DEV)
    norm = torch.linalg.vector_norm(norms).reshape(1)
    if c["op"] == "grads":
        return {"norm": norm, "norms": norms}
    if c["into"] == "tiles":
        factor = min(1.0, s["most"] / float(norm))
        B, tiles = c["B"], torch.zeros((_tile_count(c), c["B"], c["B"]), dtype=torch.float64, device=DEV)
        at = 0
        for g in s["grads"]:
            for i in range(0, g.shape[0], B):
                for j in range(0, g.shape[1], B):
                    part = g[i:i + B, j:j + B].double() * factor
                    tiles[at, :part.shape[0], :part.shape[1]] = part
                    at += 1
        return {"norm": norm, "tiles": tiles}
    factor = min(1.0, s["most"] / float(s["norm"]))
    flat = {t: f.double() for t, f in s["flat"].items()}
    for g, (r, k, ld, t) in zip(s["grads"], _shapes(c)):
        flat[t].as_strided(g.shape, g.stride(), g.storage_offset()).mul_(factor)
    return flat
