"""The launch rules at the sizes of tests/test_gpu_mixers_long.py (CPU only): the rules'
own code, compiled for the host, says that those sizes run the steady states."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_ssd_scan_b200", "csrc")
SMS = 148


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def function(text, head):
    """A function or struct from its head to the brace that ends it."""
    i = text.index(head)
    return text[i:re.compile(r"^\};?$", re.M).search(text, i).end()] + "\n"


def constant(text, name):
    return re.search(r"constexpr \w+ %s = [^;]*;" % name, text).group(0) + "\n"


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    conv, rope = source("conv1d_bwd.cu"), source("qk_norm_rope.cu")
    code = "#include <algorithm>\n#include <cstdint>\n#include <cstdio>\n#include <cstdlib>\n"
    code += "namespace conv {\n" + "".join(constant(conv, n) for n in ("NW", "CPW", "kSegUnit", "kPerSm", "kRing"))
    code += function(conv, "struct ConvGrid {") + function(conv, "ConvGrid conv_grid(") + "}\n"
    code += "namespace rope {\n" + constant(rope, "TPB") + constant(rope, "kBwdCtas")
    code += "".join(function(rope, h) for h in ("int lanes_per_unit(", "int tile_tokens(", "int bwd_tile_tokens("))
    code += r"""}
    int main(int argc, char** argv) {
        int64_t v[8] = {};
        for (int i = 2; i < argc; ++i) v[i - 2] = std::atoll(argv[i]);
        if (argv[1][0] == 'c') {  // batch, seqlen, channels
            const conv::ConvGrid g = conv::conv_grid(v[0], v[1], v[2]);
            std::printf("%lld %lld %d\n", (long long)g.seg, (long long)g.nseg, conv::kRing);
        } else {  // tokens, heads of q and k, vector length, headdim, rot_dim, SMs
            const int lpu = rope::lanes_per_unit(v[3], v[4], v[5]);
            const int64_t heads = v[1] + v[2], cq = rope::kBwdCtas * v[1] / heads, ck = rope::kBwdCtas - cq;
            const int64_t slots = 3 * v[6], tile = rope::tile_tokens(v[0], heads, lpu, v[5], slots);
            const int64_t tq = rope::bwd_tile_tokens(v[0], v[1], lpu, v[5], cq);
            const int64_t tk = v[2] ? rope::bwd_tile_tokens(v[0], v[2], lpu, v[5], ck) : 0;
            std::printf("%lld %lld %lld %lld %lld %lld\n", (long long)tile, (long long)slots, (long long)tq,
                        (long long)cq, (long long)tk, (long long)ck);
        }
    }
    """
    d = tmp_path_factory.mktemp("rules")
    (d / "r.cpp").write_text(code)
    subprocess.check_call(["g++", "-O1", "-std=c++17", str(d / "r.cpp"), "-o", str(d / "r")])
    return lambda *a: [int(x) for x in subprocess.check_output([str(d / "r")] + [str(x) for x in a]).split()]


@pytest.mark.parametrize("b,L,C,batch", [(8, 1500, 2304, 16), (8, 1111, 2304, 16), (8, 1501, 1536, 8)])
def test_conv_segments_outlast_the_ring(rules, b, L, C, batch):
    seg, nseg, ring = rules("c", b, L, C)
    assert seg >= (ring + 2) * batch and nseg > 1, (seg, nseg, ring)


@pytest.mark.parametrize("b,L,hq,hk,n,D,R", [(1, 20011, 8, 8, 8, 128, 128), (3, 20011, 5, 1, 4, 64, 32),
                                             (2, 5003, 32, 8, 8, 64, 64), (1, 20011, 3, 0, 4, 256, 64)])
def test_head_norm_ctas_take_several_tiles(rules, b, L, hq, hk, n, D, R):
    """More tiles than CTAs at once, and a last tile that is short, on one side at
    least."""
    tile, slots, tq, cq, tk, ck = rules("r", b * L, hq, hk, n, D, R, SMS)
    tokens = b * L
    assert -(-tokens // tile) > slots and -(-tokens // tq) > cq and (not tk or -(-tokens // tk) > ck)
    assert any(t and tokens % t for t in (tile, tq, tk))


@pytest.mark.parametrize("b,C", [(257, 5120), (258, 5120), (513, 2560), (1027, 1544)])
def test_decode_step_takes_four_rows_per_thread(b, C):
    text = source("gated_scan.cu")
    threads = int(re.search(r"kUpdateThreads = (\d+);", text).group(1))
    rule = re.search(r"return ctas >= (\d+) \* device_sms\(\)", text)
    assert -(-(C // 4) // threads) * -(-b // 4) >= int(rule.group(1)) * SMS
