"""Calls that need more threads than one launch holds (2^32): every output is written."""
import pytest
import torch

import matrix_inverse_roots_amd as dash

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def free_memory():
    torch.cuda.empty_cache()
    if torch.cuda.get_device_properties(0).total_memory < 100 * 2**30:
        pytest.skip("needs 100 GiB")
    yield
    torch.cuda.empty_cache()


def test_frobenius_scale_of_many_blocks():
    N, B = (1 << 22) + 3, 64
    A = torch.ones((N, B, B), device=DEV)
    A[-1] = 2.0
    s = torch.full((N,), -1.0, device=DEV)
    dash.dash_scale(A, N, B, dash.DASH_SCALE_FROBENIUS, dash.DASH_FP32, 0, 0, None, s, None)
    assert bool((s[:-1] == 64.0).all()) and float(s[-1]) == 128.0


def test_pieces_of_a_long_vector():
    n, B = (1 << 32) + 100, 64
    v = torch.ones(n, device=DEV)
    v[-1] = 3.0
    pieces = torch.full((-(-n // B), B), -1.0, device=DEV)
    dash.dash_stack_vec([v], B, pieces)
    flat = pieces.view(-1)
    assert float(flat[n - 1]) == 3.0 and not flat[n:].any()
    flat[n - 1] = 1.0
    assert bool((flat[:n] == 1.0).all())
    flat.fill_(5.0)
    dash.dash_unstack_vec(pieces, B, [v])
    assert bool((v == 5.0).all())
