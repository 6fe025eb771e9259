"""dash_apply in the least workspace it takes: the intermediate and its own bounds, whatever other calls of
the same operation's size need."""
import pytest
import torch

import matrix_inverse_roots_amd as dash
from test_mx_workspaces import apply_bytes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("prec", [dash.DASH_FP32, dash.DASH_FP32_SPLIT, dash.DASH_FP32_SPLIT16])
@pytest.mark.parametrize("N,B", [(100, 64), (7, 192), (40, 256), (9, 512), (5, 1024)])
def test_apply_in_its_own_workspace(N, B, prec):
    gen = torch.Generator(device=DEV).manual_seed(N)
    XL, XR, G = (torch.randn((N, B, B), generator=gen, device=DEV) for _ in range(3))
    U, want = torch.empty_like(G), torch.empty_like(G)
    n = apply_bytes(N, B)
    buf = torch.full((n + 4096,), 77, dtype=torch.uint8, device=DEV)
    dash.dash_apply_prec(XL, XR, G, N, B, prec, U, ws=buf[:n])
    dash.dash_apply_prec(XL, XR, G, N, B, prec, want, ws=torch.empty(n + (1 << 20), dtype=torch.uint8, device=DEV))
    assert torch.equal(U, want) and bool((buf[n:] == 77).all())
