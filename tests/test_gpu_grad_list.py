"""A list of gradients that is described once, whose tensors then change: no call reads or writes memory that is not
theirs."""
import pytest
import torch

import matrix_inverse_roots_amd as dash
from gpu_helpers import DEV
from test_gpu_norm import randn

pytestmark = pytest.mark.gpu


def test_changed_tensors_are_refused():
    ts = [randn(i, 64, 128) for i in range(4)]
    lst = dash.grad_list(ts)
    total, G = torch.empty(1, device=DEV), torch.empty((9, 64, 64), device=DEV)
    ws = dash.grad_norm_workspace(lst, device=DEV)
    dash.dash_grad_norm(lst, total, ws=ws)
    v = float(total)
    old = ts[2].data
    ts[2].data = randn(9, 64, 128)
    before = [t.clone() for t in (*ts, old)]
    for call in (lambda: dash.dash_grad_norm(lst, total, ws=ws), lambda: dash.dash_grad_clip(lst, total, 0.5 * v),
                 lambda: dash.dash_stack_clip(lst, 64, total, 0.5 * v, G), lambda: dash.grad_norm_workspace(lst)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert float(total) == v and all(torch.equal(a, b) for a, b in zip((*ts, old), before))
    again = dash.grad_list(ts)
    dash.dash_grad_clip(again, total, 0.5 * v)
    assert all(torch.equal(t, b * 0.5) for t, b in zip(ts, before))


def test_a_tensor_that_shrank():
    t = randn(3, 256, 128)
    lst = dash.grad_list([t])
    total = torch.full((1,), 4.0, device=DEV)
    G = torch.full((8, 64, 64), 7.0, device=DEV)
    dash.dash_stack_clip(lst, 64, total, 1.0, G)
    assert torch.equal(G[1], t[:64, 64:] * 0.25)
    t.resize_(64, 128)
    small = torch.full((2, 64, 64), 7.0, device=DEV)
    with pytest.raises(ValueError):
        dash.dash_stack_clip(lst, 64, total, 1.0, small)
    dash.dash_stack_clip(dash.grad_list([t]), 64, total, 1.0, small)
    assert torch.equal(small, G[:2])
