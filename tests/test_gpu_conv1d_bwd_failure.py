"""The bounded wait of the convolution's gradient: its first warp leaves one batch of
tokens out (ssd_debug_set_withhold), the wait for it gives up after about a second,
and the status call reports SSD_ERR_TIMEOUT once; the same process then runs the call
normally and gets the values from before.  In a child process with a time limit;
nothing faults or traps."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys, torch
sys.path.insert(0, ROOT)
import mamba_ssd_scan_b200 as ssd
g = torch.Generator(device="cuda").manual_seed(5)
rn = lambda *s: torch.randn(s, generator=g, device="cuda")
x, dy = (rn(8, 1500, 2304).to(getattr(torch, DTYPE)) for _ in range(2))
w, st = rn(2304, 4), rn(8, 2304, 3)
run = lambda: ssd.ssd_causal_conv1d_bwd(x, w, dy, init_state=st)
want = run()
assert ssd.ssd_conv1d_check_status() == 0
ssd.ssd_debug_set_withhold(ssd.SSD_DEBUG_CONV_TILE, BATCH)
run()
st_ = ssd.ssd_conv1d_check_status()
assert st_ == 4, f"expected SSD_ERR_TIMEOUT (4), got {st_}"
assert ssd.ssd_conv1d_check_status() == 0
ssd.ssd_debug_set_withhold(ssd.SSD_DEBUG_CONV_TILE, -1)
again = run()
assert ssd.ssd_conv1d_check_status() == 0
assert all(torch.equal(want[k], again[k]) for k in want)
print("TIMEOUT-OK")
"""


@pytest.mark.parametrize("dtype,batch", [("bfloat16", 0), ("bfloat16", 1), ("float32", 2)])
def test_a_withheld_batch_times_out(dtype, batch):
    """The first batch and later ones, whose segment has stores on their way by then."""
    code = f"ROOT = {ROOT!r}\nDTYPE = {dtype!r}\nBATCH = {batch}\n" + SCRIPT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and "TIMEOUT-OK" in r.stdout, r.stdout + r.stderr
