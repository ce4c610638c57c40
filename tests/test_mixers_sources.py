"""Rules of the kernels' sources that no run can show to be broken without hanging or
racing on the GPU (CPU only)."""
import os
import re
import subprocess

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


def test_a_check_takes_nothing_away():
    """A status check that read a word and then cleared it with a second copy would
    lose what a call on another stream reports between the two: the checks write no
    word of the device."""
    names = [n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h"))]
    assert any("cudaMemcpyFromSymbolAsync" in source(n) for n in names)
    assert not [n for n in names if "cudaMemcpyToSymbolAsync" in source(n)]


HARNESS = r"""
#include <cassert>
#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
static uint32_t word;          // the device's
static void (*meanwhile)();    // what other streams do while the copy is waited for
#define cudaGetDevice(p) (*(p) = 0, cudaSuccess)
#define cudaMemcpyFromSymbolAsync(dst, sym, n, off, kind, s) (std::memcpy(dst, &(sym), n), cudaSuccess)
#define cudaStreamSynchronize(s) (meanwhile ? (meanwhile(), cudaSuccess) : cudaSuccess)
#include "internal.cuh"
int main() {
    static ssd::GaveUp g;
    int v = -1;
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == 0);
    word += 3;
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == SSD_ERR_TIMEOUT);
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == 0);
    word += 1;
    meanwhile = [] { ++word; };  // after the copy: the next check's
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == SSD_ERR_TIMEOUT);
    meanwhile = nullptr;
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == SSD_ERR_TIMEOUT);
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == 0);
    word = 0xffffffffu;          // the count wraps
    g.seen[0] = word;
    word += 2;
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == SSD_ERR_TIMEOUT);
    assert(g.take(word, &v, nullptr) == cudaSuccess && v == 0);
    return 0;
}
"""


def test_every_wait_that_gave_up_is_reported(tmp_path):
    """The check itself, on the host, with the device's word as a variable."""
    from mamba_ssd_scan_b200 import build
    (tmp_path / "g.cu").write_text(HARNESS)
    exe = str(tmp_path / "g")
    subprocess.check_call([build.nvcc()] + build.NVCC_FLAGS + [str(tmp_path / "g.cu"), "-o", exe])
    subprocess.check_call([exe])
