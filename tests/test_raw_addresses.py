"""The binding on raw device addresses and an explicit stream, in a program without torch (no GPU: every call
is refused by the library before a launch)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["torch"] = None  # any import of it raises
import matrix_inverse_roots_amd as dash
P = [(i + 1) << 24 for i in range(8)]

class Ws:
    def data_ptr(self): return P[7]
    def numel(self): return 256
    def element_size(self): return 1

for want, fn, args, kw in (
    (3, dash.dash_apply, (P[0], P[1], P[2], 4, 64, P[3]), {"ws": None}),
    (3, dash.dash_apply, (P[0], P[1], P[2], 4, 64, P[3]), {"ws": Ws()}),
    (1, dash.dash_update_stats, (P[0], 4, 64, 1.5, P[1]), {}),
    (2, dash.dash_inverse_root_ndb, (P[0], P[1], 4, 96, 5, 5, P[2]), {"ws": Ws()}),
    (1, dash.dash_mx_quantize, (P[0], 1, 64, 64, dash.DASH_MX_E4M3), {}),
    (1, dash.dash_mx_dequantize, (P[0], P[1], 1, 64, 64, 7, P[2]), {}),
    (1, dash.dash_update_stats_mx, (P[0], P[1], P[2], P[3], 0, 64, 1, 0.5, P[4]), {}),
    (3, dash.dash_apply_mx, (P[0], P[1], P[2], P[3], P[4], 4, 64, 1, P[5]), {"ws": Ws()}),
    (2, dash.dash_grad_stack_mx, (P[0], P[1], P[2], 1, 8, 0, 64, 64, P[3]), {"ldy": 64}),
):
    try:
        fn(*args, stream=0, **kw)
    except dash.DashError as e:
        assert e.status == want, (fn.__name__, e.status)
    else:
        raise AssertionError(fn.__name__)
assert dash.dash_grad_stack_mx_workspace(100000, 64, 64, dash.DASH_FP32) > 0
print("reached the library")
"""


def test_raw_addresses_need_no_torch():
    p = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "reached the library" in p.stdout, p.stderr
