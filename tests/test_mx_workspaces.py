"""Host-side tests of the update's and the gradient tiles' workspace sizes (no GPU): nothing is launched."""
import numpy as np
import pytest
import torch

import matrix_inverse_roots_amd as dash
from test_mx_abi import E2, E4, P, WS, Ws, status


def up(n):
    return -(-n // 256) * 256


def apply_bytes(N, B):
    """dash_apply: T, a bound per block of XL, G and XR, and T's per-wave maxima."""
    return up(4 * N * B * B) + 3 * up(4 * N) + up(4 * N * 8 * (B // 256) ** 2)


def test_the_sizes_that_dash_apply_takes():
    assert apply_bytes(1536, 1024) == 6443255808 and apply_bytes(100, 64) == 1639936
    for N, B in ((1536, 1024), (100, 64), (3, 192), (50, 448)):
        reported = dash.dash_workspace_size(dash.DASH_OP_APPLY, N, B)
        assert reported >= apply_bytes(N, B)  # (dash_apply_mx's bounds can take more)
        for prec in (dash.DASH_FP32, dash.DASH_FP32_SPLIT, dash.DASH_FP32_SPLIT16):
            assert status(dash.dash_apply_prec, P[0], P[1], P[2], N, B, prec, P[3],
                          ws=Ws(P[8], apply_bytes(N, B) - 1)) == WS
        # and the microscaled update wants all of its own: T and more than one bound per block
        assert status(dash.dash_apply_mx, P[0], P[1], P[2], P[3], P[4], N, B, E2, P[5],
                      ws=Ws(P[8], up(4 * N * B * B) + 3 * up(4 * N) - 1)) == WS


def test_gradient_workspace_is_for_its_token_count():
    """The size can fall as T grows: a workspace for one T alone is refused by another that needs more, and one
    for several serves each."""
    size = lambda T: dash.dash_grad_stack_mx_workspace(T, 256, 192, dash.DASH_BF16)
    make = lambda T: dash.grad_stack_mx_workspace(T, 256, 192, torch.bfloat16, device="cpu")
    sizes = {T: size(T) for T in range(1, 4097)}
    for T in range(1, 4096):
        if sizes[T] > sizes[4096]:
            assert status(dash.dash_grad_stack_mx, P[0], P[1], P[2], E4, T, 256, 192, 64, P[3], type=dash.DASH_BF16,
                          ws=Ws(P[8], sizes[4096])) == WS
            break
    counts = [100, 1024, 2000, 4096]
    for T in (counts, tuple(counts), iter(counts), np.array(counts), torch.tensor(counts)):
        assert make(T).numel() == max(sizes[t] for t in counts) > 0
    assert make(range(1, 4097)).numel() == max(sizes.values())
    for T in (4096, np.int64(4096), torch.tensor(4096)):
        assert make(T).numel() == sizes[4096]
    assert make([1, 2]) is None and make(1) is None
    for T in ([], 1.5, [1.5]):
        with pytest.raises((TypeError, ValueError)):
            make(T)
