"""Codes of rows of any size, at elements next to the borders between codes.

Each column's gain is the fp32 number for which y = h rstd gain comes nearest to some border of the format, but not
nearer than 2^-44 of it: of the format's borders the nearest such one is some 2^-28 to 2^-32 away, of thousands of
columns some are 2^-40 away.  The reference forms y in 64 bits with an exact sum of squares, within 2^-50; the call
knows rstd to 48 bits, so that every code is decided."""
import math

import numpy as np
import pytest
import torch

import matrix_inverse_roots_amd as dash
import mx_ref as ref
from gpu_helpers import DEV
from test_gpu_norm import FMTS, IDS, NAMES, norm

pytestmark = pytest.mark.gpu


def row_next_to_borders(n, size, fmt, dtype, with_res, seed):
    """(x, res, gain, y in 64 bits) of one row whose elements are within a factor of some 8 of `size`."""
    rng = np.random.default_rng(seed)
    sign = rng.choice([-1.0, 1.0], n)
    x = torch.tensor(size * rng.uniform(0.5, 2.0, n) * sign)[None].to(dtype)
    res = torch.tensor(0.377 * size * rng.uniform(0.5, 2.0, n) * sign)[None].to(dtype) if with_res else None
    h = (x.double() + (res.double() if with_res else 0))[0].numpy()  # (exact)
    t = h / math.sqrt(math.fsum(h * h) / n)
    top, table = ref.TOP[fmt], ref.grid(fmt)
    mid = (table[1:] + table[:-1]) / 2
    gain = (mid[:, None] / np.abs(t)).astype(np.float32)
    off = np.abs(gain.astype(np.float64) * np.abs(t) / mid[:, None] - 1)
    off[off < 2.0**-44] = 1.0
    gain = gain[np.argmin(off, 0), np.arange(n)]
    gain[::32] = 0.99 * top / np.abs(t[::32])  # (above every border: the scale is 1)
    return x.to(DEV), None if res is None else res.to(DEV), torch.tensor(gain, device=DEV), (t * gain)[None]


def check(n, size, fmt, dtype, with_res, seed):
    x, res, gain, y = row_next_to_borders(n, size, fmt, dtype, with_res, seed)
    _, _, codes, scales, _ = norm(x, res, gain, fmt, eps=0.0)
    want, byte = ref.quantize(y, fmt)
    wrong = ref.unpack(codes.cpu().numpy()[0], fmt) != want
    assert np.array_equal(scales.cpu().numpy()[0], byte), (size, with_res)
    assert not wrong.any(), (size, with_res, int(wrong.sum()))


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("n", [7, 1000, 4096, 8208, 33024])
def test_what_a_sum_of_fp32_elements_loses(n, fmt):
    """x + res rounded to fp32 is off by up to 2^-24; rstd is that of the sums themselves."""
    for i, size in enumerate((1e-36, 1e-30, 1e-21, 1e-19, 1e-10, 1.0, 1e10, 1e23, 1e28)):
        check(n, size, fmt, torch.float32, True, 100 * n + i)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=NAMES.get)
@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("n", [7, 1000, 4096, 8208, 33024])
def test_rows_of_any_size(n, fmt, dtype):
    """rstd down to fp32's least normal numbers."""
    for i, size in enumerate((1e-36, 1e-20, 1.0, 1e20, 2.0**105, 2.0**112, 2.0**118, 2.0**122, 2.0**124)):
        for with_res in (False, True):
            check(n, size, fmt, dtype, with_res, 100 * n + 20 + i)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=NAMES.get)
@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("n", [1, 3, 7, 49, 1000, 4096, 8208, 33024])
def test_elements_on_borders(n, fmt, dtype):
    """Rows of one magnitude, for which y = +-gain, and gains on the borders between codes: to the even code."""
    table = ref.grid(fmt)
    mid = (table[1:] + table[:-1]) / 2
    rng = np.random.default_rng(n)
    T = 50
    gain = rng.choice(mid, n)
    gain[::32] = mid[-1]
    size = torch.tensor(rng.choice((1e-30, 0.1, 1.0, 77.0, 1e20), T) * rng.uniform(0.5, 2, T))[:, None].to(dtype)
    sign = torch.tensor(rng.choice([-1.0, 1.0], (T, n))).to(dtype)
    want, byte = ref.quantize(sign.double().numpy() * gain, fmt)
    for res in (None, size * sign * 0.375):
        x = (size * sign).to(DEV)
        _, _, codes, scales, _ = norm(x, None if res is None else res.to(DEV), torch.tensor(gain).float().to(DEV), fmt,
                                      eps=0.0)
        assert np.array_equal(scales.cpu().numpy()[0], byte)
        wrong = ref.unpack(codes.cpu().numpy()[0], fmt) != want
        assert not wrong.any(), (res is None, int(wrong.sum()))


@pytest.mark.parametrize("fmt", FMTS, ids=IDS)
@pytest.mark.parametrize("n", [2, 7, 8, 263, 33000])
def test_sums_of_16_bit_elements(n, fmt):
    """1 + 2^-30 is 1 in fp32, so that y = +-gain lies on its border in rows of any length."""
    table = ref.grid(fmt)
    mid = (table[1:] + table[:-1]) / 2
    rng = np.random.default_rng(n)
    gain, sign = rng.choice(mid, n), torch.tensor(rng.choice([-1.0, 1.0], (20, n)))
    gain[::32] = mid[-1]
    res = (2.0**-30 * torch.tensor(rng.choice([-1.0, 0.0, 1.0], (20, n)))).to(DEV, torch.bfloat16)
    want, byte = ref.quantize(sign.numpy() * gain, fmt)
    _, _, codes, scales, _ = norm(sign.to(DEV, torch.bfloat16), res, torch.tensor(gain).float().to(DEV), fmt, eps=0.0)
    assert np.array_equal(scales.cpu().numpy()[0], byte)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()[0], fmt), want)
