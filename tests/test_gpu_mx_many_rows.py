"""Quantisation and back over more workgroups than one launch can hold (2^32 threads): every row is written."""
import pytest
import torch

import matrix_inverse_roots_amd as dash

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FMT = dash.DASH_MX_E2M1  # one element of a group: 16 bytes of codes; 1.0 is 4 2^-2: code 6, scale byte 125


def test_many_short_rows():
    """2^31 + 130 rows of one element: 64 (fp32) or 128 rows to a workgroup."""
    N, rows = 2, (1 << 30) + 65
    if torch.cuda.get_device_properties(0).total_memory < 80 * 2**30:
        pytest.skip("needs 80 GiB")
    x = torch.ones((N, rows, 1), device=DEV)
    x[1, -1] = -6.0
    codes = torch.full((N, rows, 16), 0xFF, dtype=torch.uint8, device=DEV)
    scales = torch.full((N, rows, 1), 0xFF, dtype=torch.uint8, device=DEV)
    dash.dash_mx_quantize(x, N, rows, 1, FMT, codes, scales)
    assert int(scales[1, -1]) == 127 and codes[1, -1].tolist() == [15] + [0] * 15
    scales[1, -1], codes[1, -1, 0] = 125, 6
    assert bool((scales == 125).all())
    assert bool((codes.view(torch.int64)[..., 0] == 6).all()) and not bool(codes.view(torch.int64)[..., 1].any())
    del x
    v = torch.zeros((N, rows, 1), dtype=torch.bfloat16, device=DEV)
    codes[1, -1, 0] = 15
    dash.dash_mx_dequantize(codes, scales, N, rows, 1, FMT, v)
    assert float(v[1, -1]) == -1.5
    v[1, -1] = 1.0
    assert bool((v == 1.0).all())


@pytest.mark.parametrize("sides", ["cols", "both"])
def test_many_small_matrices(sides):
    """A workgroup per 64 x 64 of each matrix."""
    N = (1 << 24) + 77
    x = torch.ones((N, 1, 1), device=DEV)
    pairs = [[torch.full((N, 1, n), 0xFF, dtype=torch.uint8, device=DEV) for n in (16, 1)] for _ in range(2)]
    rows = pairs[0] if sides == "both" else (None, None)
    diag = torch.zeros((N, 1), device=DEV)
    dash.dash_mx_quantize(x, N, 1, 1, FMT, *rows, *pairs[-1])
    for codes, scales in pairs if sides == "both" else pairs[-1:]:
        assert bool((scales == 125).all())
        assert bool((codes.view(torch.int64)[..., 0] == 6).all()) and not bool(codes.view(torch.int64)[..., 1].any())
    dash.dash_mx_quantize(x, N, 1, 1, FMT, *rows, *pairs[-1], diag=diag)
    assert bool((diag == 1.0).all()) and bool((pairs[-1][1] == 0).all()) and not bool(pairs[-1][0].any())
