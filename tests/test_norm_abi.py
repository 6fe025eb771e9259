"""Host-side tests of the norm, its gradient, the gradient norm and clipping (no GPU): bad arguments are
refused before any launch."""
import ctypes
import itertools

import pytest
import torch

import matrix_inverse_roots_amd as dash
from matrix_inverse_roots_amd import _lib
from test_mx_abi import INVALID, P, SHAPE, WS, Ws, status

BF16, FP32 = dash.DASH_BF16, dash.DASH_FP32
NAN, INF = float("nan"), float("inf")


def norm(x=P[0], T=8, n=64, eps=1e-5, **kw):
    return status(dash.dash_rmsnorm, x, T, n, eps, **kw)


def test_norm_refusals():
    out = dict(codes=P[1], scales=P[2])
    assert norm(None, **out) == INVALID
    assert norm() == INVALID  # no output
    assert norm(codes=P[1]) == INVALID and norm(scales=P[2]) == INVALID  # half a pair
    assert norm(codes=P[1] + 8, scales=P[2]) == INVALID
    assert norm(P[0] + 2, **out) == INVALID  # fp32 misaligned
    assert norm(P[0] + 1, type=BF16, **out) == INVALID
    assert norm(res=P[3] + 2, **out) == INVALID and norm(h=P[3] + 2, **out) == INVALID
    assert norm(y=P[3] + 2, **out) == INVALID and norm(rstd=P[3] + 2, **out) == INVALID
    assert norm(gain=P[3] + 2, **out) == INVALID and norm(gain=P[3] + 1, gain_type=BF16, **out) == INVALID
    assert norm(gain=P[3], gain_type=dash.DASH_FP32_SPLIT, **out) == INVALID
    assert norm(type=dash.DASH_FP32_SPLIT16, **out) == INVALID
    assert norm(fmt=2, **out) == INVALID and norm(fmt=-1, **out) == INVALID
    for eps in (-1e-5, NAN, INF):
        assert norm(eps=eps, **out) == INVALID
    for T, n in ((-1, 64), (8, 0), (8, -4), (8, (1 << 26) + 1), (1 << 31, 64), (1 << 30, 1 << 26)):
        assert norm(T=T, n=n, **out) == SHAPE
    for ld in ("ldx", "ldr", "ldh", "ldy"):
        assert norm(res=P[3], h=P[4], y=P[5], **{ld: 63}, **out) == SHAPE, ld


def test_norm_buffers_are_apart():
    """No output shares memory with another buffer, but for h in the place of x or res."""
    names = ["x", "res", "gain", "h", "y", "codes", "scales", "rstd"]
    for a, b in itertools.combinations(range(8), 2):
        if names[a] in ("x", "res", "gain") and names[b] in ("res", "gain"):
            continue  # (two inputs)
        if names[b] == "h" and names[a] in ("x", "res"):
            continue
        p = dict(zip(names, P))
        p[names[b]] = p[names[a]]
        assert norm(**p) == INVALID, (names[a], names[b])
    size = 8 * 64 * 4
    out = dict(codes=P[5], scales=P[6])
    assert norm(y=P[0] + size - 4, **out) == INVALID and norm(y=P[0] - size + 16, **out) == INVALID
    assert norm(h=P[0], ldh=65, **out) == INVALID  # x's place in another pitch
    # half of a wider buffer's columns: too few, or its own
    assert norm(y=P[0] + 63 * 4, ldx=128, ldy=128, **out) == INVALID
    assert norm(y=P[0] + 65 * 4, ldx=128, ldy=128, **out) == INVALID


def back(dy=P[0], h=P[1], rstd=P[2], T=8, n=64, dx=P[3], **kw):
    return status(dash.dash_rmsnorm_backward, dy, h, rstd, T, n, dx, **kw)


def test_gradient_refusals():
    for name in ("dy", "h", "rstd", "dx"):
        assert back(**{name: None}) == INVALID, name
    for name in ("dy", "h", "rstd", "dx", "dh", "gain", "dgain"):
        assert back(**{name: P[7] + 2}) == INVALID, name
    assert back(type=dash.DASH_FP32_SPLIT) == INVALID
    for T, n in ((-1, 64), (8, 0), (8, (1 << 26) + 1), (1 << 31, 64)):
        assert back(T=T, n=n) == SHAPE
    for ld in ("lddy", "ldh", "lddh", "lddx"):
        assert back(dh=P[4], **{ld: 63}) == SHAPE, ld
    need = dash.dash_rmsnorm_backward_workspace(8, 64)
    assert need > 0
    assert back(dgain=P[5]) == WS
    assert back(dgain=P[5], ws=Ws(P[6], need - 1)) == WS and back(dgain=P[5], ws=Ws(P[6] + 16, need)) == WS
    assert back(dgain=P[5], ws=Ws(P[0], need)) == WS  # over dy
    lib = dash.library()
    assert lib.dash_rmsnorm_backward(P[0], 64, P[1], 64, None, 64, FP32, None, FP32, P[2], 8, 64, P[3], 64, None, 2,
                                     None, 0, None) == INVALID
    assert lib.dash_rmsnorm_backward_workspace(8, 64, None) == INVALID
    for T, n in ((-1, 64), (8, 0)):
        with pytest.raises(dash.DashError):
            dash.dash_rmsnorm_backward_workspace(T, n)
    # the size for one T serves any smaller one
    for n in (1, 263, 2048, 1 << 20):
        sizes = [dash.dash_rmsnorm_backward_workspace(T, n) for T in (0, 1, 2, 500, 512, 513, 4000, 1 << 20)]
        assert sizes == sorted(sizes)


def test_gradient_buffers_are_apart():
    names = ["dy", "h", "rstd", "dh", "gain", "dx", "dgain"]
    ws = Ws(P[8], dash.dash_rmsnorm_backward_workspace(8, 64))
    for a, b in itertools.combinations(range(7), 2):
        if names[b] not in ("dx", "dgain") or (names[b] == "dx" and names[a] in ("dy", "dh")):
            continue
        p = dict(zip(names, P))
        p[names[b]] = p[names[a]]
        assert back(ws=ws, **p) == INVALID, (names[a], names[b])


def tensors(*specs):
    arr = (_lib.DashTensor * len(specs))()
    for i, s in enumerate(specs):
        arr[i] = s
    return arr


GOOD = (P[0], 8, 64, 64, FP32)


def grads_statuses(arr, n):
    lib = dash.library()
    size = ctypes.c_size_t()
    return {lib.dash_grad_norm_workspace(arr, n, ctypes.byref(size)),
            lib.dash_grad_norm(arr, n, P[9], None, P[10], 1 << 20, None),
            lib.dash_grad_clip(arr, n, P[9], 1.0, None)}


def test_gradient_descriptors():
    for bad, why in (((None, 8, 64, 64, FP32), INVALID), ((P[0] + 2, 8, 64, 64, FP32), INVALID),
                     ((P[0] + 1, 8, 64, 64, BF16), INVALID), ((P[0], 8, 64, 64, dash.DASH_FP32_SPLIT), INVALID),
                     ((P[0], 8, 64, 64, 17), INVALID), ((P[0], -1, 64, 64, FP32), SHAPE),
                     ((P[0], 8, -1, 64, FP32), SHAPE), ((P[0], 8, 64, 63, FP32), SHAPE),
                     ((P[0], 1, 1 << 45, 1 << 45, FP32), SHAPE), ((P[0], 1 << 32, 8, 9, FP32), SHAPE),
                     ((P[0], 1 << 30, 1 << 16, 1 << 16, FP32), SHAPE), ((P[0], 1 << 62, 1 << 62, 1 << 62, FP32), SHAPE)):
        assert grads_statuses(tensors(bad), 1) == {why}, bad
        assert grads_statuses(tensors((P[1], 8, 64, 64, FP32), bad), 2) == {why}, bad
    assert grads_statuses(tensors(GOOD), -1) == {INVALID} and grads_statuses(None, 1) == {INVALID}
    assert dash.library().dash_grad_norm_workspace(tensors(GOOD), 1, None) == INVALID


def test_gradient_norm_refusals():
    lib = dash.library()
    arr = tensors(GOOD, (P[1], 1, 100, 100, BF16))
    size = ctypes.c_size_t()
    assert lib.dash_grad_norm_workspace(arr, 2, ctypes.byref(size)) == 0 and size.value > 0
    need = size.value

    def f(norm, norms=None, ws=P[10], n=need):
        return lib.dash_grad_norm(arr, 2, norm, norms, ws, n, None)

    assert f(None) == INVALID and f(P[9] + 2) == INVALID and f(P[9], P[8] + 2) == INVALID
    assert f(P[9], P[9]) == INVALID and f(P[9] + 4, P[9]) == INVALID
    assert f(P[0] + 64) == INVALID and f(P[9], P[1] - 4) == INVALID  # inside a gradient
    assert f(P[9], ws=None) == WS and f(P[9], n=need - 1) == WS and f(P[9], ws=P[10] + 8) == WS
    assert f(P[10]) == WS and f(P[9], ws=P[0]) == WS


def test_the_norm_s_workspace_does_not_go_by_addresses():
    size = ctypes.c_size_t()
    for rows, cols, ld in ((1, 5, 5), (1, 4096, 4096), (1, 1 << 20, 1 << 20), (300, 257, 300), (3000, 64, 80), (1, 1 << 33,
                           1 << 33)):
        for dtype, step in ((FP32, 4), (BF16, 2)):
            got = set()
            for off in range(0, 16, step):
                arr = tensors((P[0] + off, rows, cols, ld, dtype), (P[1] + off, 1, 77, 77, dtype))
                assert dash.library().dash_grad_norm_workspace(arr, 2, ctypes.byref(size)) == 0
                got.add(size.value)
            assert len(got) == 1


def test_clip_refusals():
    lib = dash.library()
    arr = tensors(GOOD)

    def f(arr, n, norm=P[9], most=1.0):
        return lib.dash_grad_clip(arr, n, norm, most, None)

    assert f(arr, 1, None) == INVALID and f(arr, 1, P[9] + 2) == INVALID
    assert f(arr, 1, most=-1.0) == INVALID and f(arr, 1, most=NAN) == INVALID
    assert f(arr, 1, P[0] + 4) == INVALID  # the norm inside a gradient
    # gradients that share memory: the same twice, one inside another, overlapping ends, slices that meet
    wide = (P[0], 8, 64, 200, FP32)
    for other in (GOOD, (P[0] + 256, 1, 4, 4, FP32), (P[0] + 8 * 64 * 4 - 4, 1, 64, 64, FP32),
                  (P[0] - 4, 1, 2, 2, FP32), (P[0], 1, 1, 1, BF16)):
        assert f(tensors(GOOD, (P[3], 4, 4, 4, FP32), other), 3) == INVALID, other
        assert f(tensors(other, (P[3], 4, 4, 4, FP32), GOOD), 3) == INVALID, other
    for other in ((P[0] + 63 * 4, 8, 64, 200, FP32), (P[0] + 150 * 4, 8, 64, 200, FP32),
                  (P[0] + 130 * 4, 1, 71, 71, FP32), (P[0] + 3 * 800 + 63 * 4, 1, 1, 1, FP32),
                  (P[0] + 100 * 4, 8, 64, 150, FP32)):
        assert f(tensors(wide, other), 2) == INVALID, other

    def g(grads=P[0], B=64, norm=P[9], most=1.0, G=P[5], ld=64):
        return lib.dash_stack_clip((_lib.DashMat * 1)((grads, 8, 64, ld)), 1, B, norm, most, G, None)

    assert g(None) == INVALID and g(G=None) == INVALID and g(norm=None) == INVALID and g(G=P[5] + 4) == INVALID
    assert g(norm=P[9] + 1) == INVALID and g(most=-0.5) == INVALID and g(most=NAN) == INVALID
    assert g(ld=66) == INVALID and g(B=100) == SHAPE and g(norm=P[5] + 64 * 64 * 4 - 4) == INVALID
    assert lib.dash_stack_clip(None, 1, 64, P[9], 1.0, P[5], None) == INVALID
    # the stack over a gradient: at its last element, behind its first, and the other way round
    for G, ld in ((P[4] + 7 * 64 * 4 + 240, 64), (P[4] - 64 * 64 * 4 + 16, 64), (P[4], 64), (P[4] + 64 * 4, 128)):
        assert g(grads=P[4], G=G, ld=ld) == INVALID, (G - P[4], ld)


def test_host_tensors_and_other_types_are_refused():
    x = torch.zeros(8, 64)
    for call in (lambda: dash.dash_rmsnorm(x, 8, 64, 1e-5, y=P[1], stream=0),
                 lambda: dash.dash_rmsnorm_backward(P[0], x, P[2], 8, 64, P[3], stream=0),
                 lambda: dash.grad_list([x]), lambda: dash.dash_grad_norm([x], P[0], stream=0),
                 lambda: dash.dash_grad_clip([P[0]], P[0], 1.0, stream=0),
                 lambda: dash.dash_stack_clip([x], 64, P[0], 1.0, P[1], stream=0)):
        with pytest.raises(ValueError):
            call()


def test_an_empty_list_needs_no_workspace():
    assert dash.dash_grad_norm_workspace([]) == 0
    assert len(dash.grad_list([])) == 0
    dash.dash_grad_clip([], P[0], 1.0, stream=0)  # nothing to do
