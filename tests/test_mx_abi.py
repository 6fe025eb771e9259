"""Host-side tests of the microscaled calls (no GPU): bad arguments are refused before any launch, and
the plain 64-bit reference the GPU tests use agrees with the format's definition."""
import numpy as np
import pytest
import torch

import matrix_inverse_roots_amd as dash
from matrix_inverse_roots_amd import _lib
import mx_ref

P = [(i + 1) << 24 for i in range(12)]  # fake, well aligned, distinct device addresses
E2, E4 = dash.DASH_MX_E2M1, dash.DASH_MX_E4M3
INVALID, SHAPE, WS = _lib.DASH_ERR_INVALID_ARG, _lib.DASH_ERR_SHAPE, _lib.DASH_ERR_WORKSPACE


def status(fn, *args, **kw):
    with pytest.raises(dash.DashError) as e:
        fn(*args, stream=0, **kw)
    return e.value.status


class Ws:
    def __init__(self, ptr, n):
        self.ptr, self.n = ptr, n

    def data_ptr(self):
        return self.ptr

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def test_quantize_refusals():
    f = dash.dash_mx_quantize
    assert status(f, None, 1, 64, 64, E4, P[1], P[2]) == INVALID                    # no source
    assert status(f, P[0], 1, 64, 64, E4) == INVALID                                # no output
    assert status(f, P[0], 1, 64, 64, E4, P[1], None) == INVALID                    # half a pair
    assert status(f, P[0], 1, 64, 64, E4, None, P[2]) == INVALID
    assert status(f, P[0], 1, 64, 64, E4, P[1], P[2], P[3], None) == INVALID
    assert status(f, P[0], 1, 64, 64, E4, P[1] + 8, P[2]) == INVALID                # codes misaligned
    assert status(f, P[0], 1, 64, 64, E4, P[1], P[2], P[1], P[3]) == INVALID        # both into one buffer
    assert status(f, P[0], 1, 64, 64, E4, P[0], P[2]) == INVALID                    # over the source
    assert status(f, P[0] + 2, 1, 64, 64, E4, P[1], P[2]) == INVALID                # fp32 misaligned
    assert status(f, P[0], 1, 64, 64, 2, P[1], P[2]) == INVALID                     # no such format
    assert status(f, P[0], 1, 64, 64, E4, P[1], P[2], type=dash.DASH_FP32_SPLIT) == INVALID
    assert status(f, P[0], 0, 64, 64, E4, P[1], P[2]) == INVALID                    # no matrix
    for rows, cols, ld in ((0, 64, 64), (64, 0, 64), (64, 64, 63), (-1, 64, 64), (1 << 31, 64, 64)):
        assert status(f, P[0], 1, rows, cols, E4, P[1], P[2], ld=ld) == SHAPE
    assert status(f, P[0], 1 << 20, 1 << 20, 1 << 20, E4, P[1], P[2]) == SHAPE      # more than memory holds
    assert status(f, P[0], 1, 64, 65, E4, P[1], P[2], diag=P[3]) == SHAPE           # diagonal of no square
    assert status(f, P[0], 1, 64, 64, E4, P[1], P[2], diag=P[3] + 2) == INVALID


def test_dequantize_refusals():
    f = dash.dash_mx_dequantize
    assert status(f, None, P[1], 1, 64, 64, E4, P[2]) == INVALID
    assert status(f, P[0], None, 1, 64, 64, E4, P[2]) == INVALID
    assert status(f, P[0], P[1], 1, 64, 64, E4, None) == INVALID
    assert status(f, P[0] + 4, P[1], 1, 64, 64, E4, P[2]) == INVALID
    assert status(f, P[0], P[1], 1, 64, 64, E4, P[0]) == INVALID
    assert status(f, P[0], P[1], 1, 64, 64, -1, P[2]) == INVALID
    assert status(f, P[0], P[1], 1, 64, 64, E4, P[2] + 1, type=dash.DASH_BF16) == INVALID
    assert status(f, P[0], P[1], 1, 64, 64, E4, P[2], ld=32) == SHAPE
    assert status(f, P[0], P[1], 1, 64, 32, E4, P[2], diag=P[3]) == SHAPE


def test_stats_refusals():
    f = dash.dash_update_stats_mx
    assert status(f, None, P[1], P[2], P[3], 4, 64, E4, 0.9, P[4]) == INVALID
    assert status(f, P[0], None, P[2], P[3], 4, 64, E4, 0.9, P[4]) == INVALID
    assert status(f, P[0], P[1], None, P[3], 4, 64, E4, 0.9, P[4]) == INVALID
    assert status(f, P[0], P[1], P[2], None, 4, 64, E4, 0.9, P[4]) == INVALID
    assert status(f, P[0], P[1], P[2] + 8, P[3], 4, 64, E4, 0.9, P[4]) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], 4, 64, 5, 0.9, P[4]) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], 4, 64, E4, 1.5, P[4]) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], 4, 64, E4, float("nan"), P[4]) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], 0, 64, E4, 0.9, P[4]) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], 4, 64, E4, 0.9, None) == INVALID
    for B in (32, 96, 8256):
        assert status(f, P[0], P[1], P[2], P[3], 4, B, E4, 0.9, P[4]) == SHAPE


def test_apply_refusals():
    f = dash.dash_apply_mx
    n = dash.dash_workspace_size(dash.DASH_OP_APPLY, 4, 64)
    ws = Ws(P[8], n)
    assert status(f, None, P[1], P[2], P[3], P[4], 4, 64, E2, P[5], ws=ws) == INVALID
    assert status(f, P[0], P[1], P[2], None, P[4], 4, 64, E2, P[5], ws=ws) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], None, 4, 64, E2, P[5], ws=ws) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], P[4], 4, 64, E2, P[4], ws=ws) == INVALID  # U over G
    assert status(f, P[0], P[1], P[2], P[3], P[4], 4, 64, 3, P[5], ws=ws) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], P[4], 0, 64, E2, P[5], ws=ws) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], P[4], 4, 64, E2, P[5], XL_diag=P[6] + 2, ws=ws) == INVALID
    assert status(f, P[0], P[1], P[2], P[3], P[4], 4, 96, E2, P[5], ws=ws) == SHAPE
    assert status(f, P[0], P[1], P[2], P[3], P[4], 4, 64, E2, P[5]) == WS
    assert status(f, P[0], P[1], P[2], P[3], P[4], 4, 64, E2, P[5], ws=Ws(P[8], n - 1)) == WS
    assert status(f, P[0], P[1], P[2], P[3], P[4], 4, 64, E2, P[5], ws=Ws(P[8] + 16, n)) == WS


def test_grad_stack_refusals():
    f = dash.dash_grad_stack_mx
    assert status(f, None, P[1], P[2], E4, 8, 64, 64, 64, P[3]) == INVALID
    assert status(f, P[0], None, P[2], E4, 8, 64, 64, 64, P[3]) == INVALID
    assert status(f, P[0], P[1], None, E4, 8, 64, 64, 64, P[3]) == INVALID
    assert status(f, P[0], P[1], P[2], E4, 8, 64, 64, 64, None) == INVALID
    assert status(f, P[0], P[1], P[2], 9, 8, 64, 64, 64, P[3]) == INVALID
    assert status(f, P[0] + 2, P[1], P[2], E4, 8, 64, 64, 64, P[3]) == INVALID
    assert status(f, P[0], P[1], P[2], E4, 8, 64, 64, 64, P[0]) == INVALID
    assert status(f, P[0], P[1], P[2], E4, 8, 64, 64, 64, P[3], type=dash.DASH_FP32_SPLIT16) == INVALID
    for T, out, inp, ldy in ((-1, 64, 64, 64), (8, 0, 64, 64), (8, 64, 0, 64), (8, 64, 64, 63),
                             (1 << 30, 1 << 20, 64, 1 << 20)):
        assert status(f, P[0], P[1], P[2], E4, T, out, inp, 64, P[3], ldy=ldy) == SHAPE
    assert status(f, P[0], P[1], P[2], E4, 8, 64, 64, 100, P[3]) == SHAPE
    n = dash.dash_grad_stack_mx_workspace(100000, 64, 64, dash.DASH_BF16)
    assert n > 0
    args = (P[0], P[1], P[2], E4, 100000, 64, 64, 64, P[3])
    assert status(f, *args, type=dash.DASH_BF16) == WS
    assert status(f, *args, type=dash.DASH_BF16, ws=Ws(P[8], n - 1)) == WS
    assert status(f, *args, type=dash.DASH_BF16, ws=Ws(P[8] + 64, n)) == WS
    assert dash.dash_grad_stack_mx_workspace(0, 64, 64, dash.DASH_BF16) == 0
    assert dash.dash_grad_stack_mx_workspace(16, 8192, 8192, dash.DASH_FP32) == 0
    lib = dash.library()
    assert lib.dash_grad_stack_mx_workspace(8, 64, 64, dash.DASH_FP32, None) == INVALID
    with pytest.raises(dash.DashError):
        dash.dash_grad_stack_mx_workspace(8, 64, 64, dash.DASH_FP32_SPLIT)
    # accumulate is 0 or 1
    assert lib.dash_grad_stack_mx(P[0], dash.DASH_FP32, 64, P[1], P[2], E4, 8, 64, 64, 64, 2, P[3], None, 0,
                                  None) == INVALID


def test_host_tensors_are_refused():
    x = torch.zeros(64, 64)
    with pytest.raises(ValueError):
        dash.dash_mx_quantize(x, 1, 64, 64, E4, P[1], P[2], stream=0)
    with pytest.raises(ValueError):
        dash.dash_grad_stack_mx(x, P[1], P[2], E4, 64, 64, 64, 64, P[3], stream=0)


@pytest.mark.parametrize("fmt,top,code", [(E2, 6.0, 7), (E4, 448.0, 126)])
def test_reference_format(fmt, top, code):
    """The largest value keeps e = 0, the next fp32 above it doubles the scale; ties go to even codes."""
    x = np.zeros((1, 32))
    x[0, 0] = top
    c, s = mx_ref.quantize(x, fmt)
    assert c[0, 0] == code and s[0, 0] == 127
    x[0, 0] = np.nextafter(np.float32(top), np.float32(np.inf))
    c, s = mx_ref.quantize(x, fmt)
    assert s[0, 0] == 128
    t = mx_ref.grid(fmt)
    x = np.full((1, 32), top)
    x[0, 1:7] = (t[1:7] + t[:6]) / 2
    c, _ = mx_ref.quantize(x, fmt)
    assert np.all(c[0, 1:7] % 2 == 0)
    packed = mx_ref.pack(c, fmt)
    assert np.array_equal(mx_ref.unpack(packed, fmt), c)
    v = mx_ref.values(packed, np.full((1, 1), 127), 32, fmt)
    assert np.array_equal(v[0], t[c[0]])
    x[0, 3] = np.inf
    c, s = mx_ref.quantize(x, fmt)
    assert s[0, 0] == 255 and not c.any()
    c, s = mx_ref.quantize(np.zeros((1, 5)), fmt)
    assert s[0, 0] == 0 and not c.any() and c.shape == (1, 32)


def test_calls_run_on_their_tensors_device(monkeypatch):
    """A launch whose tensors live on another device than the current one makes theirs current."""
    a = _lib._Args("call")
    entered = []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *exc):
            entered.append(None)

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    a.device, a.index = torch.device("cuda:1"), 1
    a.run(lambda: entered.append("ran") or 0)
    assert entered == [torch.device("cuda:1"), "ran", None]
    a.device, a.index = torch.device("cuda:0"), 0
    del entered[:]
    a.run(lambda: entered.append("ran") or 0)
    assert entered == ["ran"]
    with pytest.raises(dash.DashError) as e:
        a.run(lambda: INVALID)
    assert e.value.status == INVALID
