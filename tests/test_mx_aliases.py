"""Host-side tests (no GPU): a microscaled call whose output is another of its buffers is refused."""
import itertools

import matrix_inverse_roots_amd as dash
from test_mx_abi import E2, E4, INVALID, P, Ws, status


def test_quantize_outputs_are_distinct():
    names = ["src", "codes", "scales", "codes_t", "scales_t", "diag"]
    for a, b in itertools.combinations(range(6), 2):
        p = list(P[:6])
        p[b] = p[a]
        assert status(dash.dash_mx_quantize, p[0], 1, 64, 64, E4, *p[1:5], diag=p[5]) == INVALID, (names[a], names[b])


def test_update_and_gradient_outputs_are_no_inputs():
    ws = Ws(P[8], dash.dash_workspace_size(dash.DASH_OP_APPLY, 4, 64))
    ins = [P[i] for i in range(7)]
    for i in range(7):
        assert status(dash.dash_apply_mx, ins[0], ins[1], ins[2], ins[3], ins[4], 4, 64, E2, ins[i], XL_diag=ins[5],
                      XR_diag=ins[6], ws=ws) == INVALID, i
    for i in range(3):
        assert status(dash.dash_grad_stack_mx, P[0], P[1], P[2], E4, 8, 64, 64, 64, P[i]) == INVALID, i
    for i in range(4):
        assert status(dash.dash_update_stats_mx, P[0], P[1], P[2], P[3], 4, 64, E4, 0.9, P[i]) == INVALID, i
    for i in range(3):
        assert status(dash.dash_mx_dequantize, P[0], P[1], 1, 64, 64, E4, P[i], diag=P[2]) == INVALID, i
