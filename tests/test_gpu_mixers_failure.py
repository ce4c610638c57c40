"""The gated recurrence's bounded waits: the first tile of a cluster withholds its
map (ssd_debug_set_withhold), the cluster's waits on it give up after about a
second, and the status call reports SSD_ERR_TIMEOUT; the same process then runs
the call normally and gets the values from before.  In a child process with a
time limit; nothing faults or traps."""
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
g = torch.Generator().manual_seed(5)
x, ga, gx, dy = (torch.randn((1, 4000, 40), generator=g).bfloat16().cuda() for _ in range(4))
decay = torch.full((40,), -4.0, device="cuda")
y, states = ssd.ssd_gated_scan(x, ga, gx, decay, return_states=True)
run = {"scan": lambda: [ssd.ssd_gated_scan(x, ga, gx, decay)],
       "bwd": lambda: list(ssd.ssd_gated_scan_bwd(x, ga, gx, decay, dy, states).values())}[MODE]
want = run()
assert ssd.ssd_gated_scan_check_status() == 0
ssd.ssd_debug_set_withhold(ssd.SSD_DEBUG_GATED_MAP, ROUND)
run()
st = ssd.ssd_gated_scan_check_status()
assert st == 4, f"expected SSD_ERR_TIMEOUT (4), got {st}"
ssd.ssd_debug_set_withhold(ssd.SSD_DEBUG_GATED_MAP, -1)
again = run()
assert ssd.ssd_gated_scan_check_status() == 0
assert all(torch.equal(a, b) for a, b in zip(want, again))
print("TIMEOUT-OK")
"""


@pytest.mark.parametrize("mode,rnd", [("scan", 0), ("scan", 2), ("bwd", 1)])
def test_withheld_map_times_out(mode, rnd):
    code = f"ROOT = {ROOT!r}\nMODE = {mode!r}\nROUND = {rnd}\n" + SCRIPT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and "TIMEOUT-OK" in r.stdout, r.stdout + r.stderr
