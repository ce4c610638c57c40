"""Rules of the kernels' sources that no run can show to be broken without hanging or
racing on the GPU (CPU only)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_ssd_scan_b200", "csrc")


def source(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_warps_join_before_an_aligned_cluster_barrier():
    """The gradient's first warp stores its sums under a condition that its lanes do
    not share (channels past the last), right before the cluster's last barrier."""
    text = source("gated_scan.cu")
    at = [m.start() for m in re.finditer(r"barrier\.cluster\.arrive[.\w]*\.aligned", text)]
    assert at
    for i in at:
        body = text[text.rindex("{\n", 0, i):i]
        assert "__syncwarp();" in body, body
