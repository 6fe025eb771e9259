"""Microscaled storage and its products from their definitions, in numpy at 64 bits (no library code)."""
import numpy as np

GROUP = 32
E2M1, E4M3 = 0, 1
TOP = {E2M1: 6.0, E4M3: 448.0}


def grid(fmt):
    """Element values by code, sign bit clear."""
    if fmt == E2M1:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    c = np.arange(127)
    return np.where(c < 8, c * 2.0**-9, (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7))


def quantize(x, fmt):
    """(codes, scale bytes) of the rows of x [..., cols]: codes one per element, padded to whole groups."""
    x = np.asarray(x, np.float64)
    g = -(-x.shape[-1] // GROUP)
    v = np.zeros((*x.shape[:-1], g * GROUP))
    v[..., : x.shape[-1]] = x
    v = v.reshape(*x.shape[:-1], g, GROUP)
    top = np.abs(v).max(-1)
    bad = ~np.isfinite(top)
    byte = np.zeros(top.shape, np.int64)
    for b in range(254, -1, -1):  # the least e (byte - 127) with top <= TOP 2^e
        byte[np.where(bad, 0, top) <= TOP[fmt] * 2.0 ** (b - 127)] = b
    y = np.where(bad[..., None], 0, v) * 2.0 ** (127.0 - byte)[..., None]
    t = grid(fmt)
    mid = (t[1:] + t[:-1]) / 2
    a = np.abs(y)
    lo = np.searchsorted(mid, a, side="left")  # a tie stays below ...
    hi = np.searchsorted(mid, a, side="right")  # ... or goes up: whichever code is even
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    code = code | (np.signbit(y).astype(np.int64) << (3 if fmt == E2M1 else 7))
    byte[bad] = 255
    return code.reshape(*x.shape[:-1], -1), byte


def pack(code, fmt):
    code = code.astype(np.uint8)
    return code if fmt == E4M3 else (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes, fmt):
    codes = np.asarray(codes)
    if fmt == E4M3:
        return codes.astype(np.int64)
    return np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).astype(np.int64)


def values(codes, scales, cols, fmt):
    """The values of packed codes and scale bytes, in 64 bits."""
    c = unpack(codes, fmt)
    t = np.concatenate((grid(fmt), [np.nan])) if fmt == E4M3 else grid(fmt)
    half = len(t)
    v = np.where(c >= half, -1.0, 1.0) * t[c % half]
    s = np.asarray(scales).astype(np.float64)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return (v * np.repeat(f, GROUP, -1))[..., :cols]


def tiles(W, B):
    r, c = -(-W.shape[0] // B), -(-W.shape[1] // B)
    P = np.zeros((r * B, c * B))
    P[: W.shape[0], : W.shape[1]] = W
    return P.reshape(r, B, c, B).transpose(0, 2, 1, 3).reshape(r * c, B, B)
