"""Host-side tests of the microscaled helpers of the binding (no GPU)."""
import pytest
import torch

import matrix_inverse_roots_amd as dash
from test_mx_abi import E2, E4


def test_buffers_of_a_known_format():
    for fmt, width in ((E2, 16), (E4, 32)):
        codes, scales = dash.mx_buffers(2, 3, 65, fmt, device="cpu")
        assert codes.shape == (2, 3, 3 * width) and scales.shape == (2, 3, 3)
    for fmt in (2, -1, None):
        with pytest.raises(ValueError):
            dash.mx_buffers(2, 3, 65, fmt, device="cpu")


def test_gradient_workspace_takes_the_element_types():
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        assert dash.grad_stack_mx_workspace(100000, 64, 64, dtype, device="cpu").dtype == torch.uint8
    for dtype in (torch.float64, torch.int32, None, dash.DASH_FP32):
        with pytest.raises(ValueError):
            dash.grad_stack_mx_workspace(100000, 64, 64, dtype, device="cpu")
