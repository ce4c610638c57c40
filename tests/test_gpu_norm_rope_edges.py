"""The head norm with the rotation where it could go wrong."""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_b200 as ssd
from oracle import mixers as om

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("adjacent", [False, True], ids=["half", "adj"])
def test_angles_of_high_frequencies_at_far_positions(adjacent):
    """Several turns per position, up to position 2^31: the angle stays within 2^-25
    of a turn (the header's figure for every frequency), beside the definition's
    own bound.  The definition's product has 64 bits: off by 2^31 * 640 * 2^-64."""
    b, L, h, D, R = 1, 64, 2, 64, 64
    g = torch.Generator().manual_seed(3)
    q = torch.randn((b, L, h, D), generator=g).to(DEV)
    f = torch.cat([torch.logspace(0, 2.8, R // 4), -torch.logspace(0, 2.8, R // 4)]).to(DEV)
    pos = torch.randint((1 << 31) - (1 << 20), 1 << 31, (b, L), generator=g)
    pos[0, ::3] *= -1
    pos = pos.to(DEV)
    ang = 2 * np.pi * 2.0 ** -25 + 2.0 ** 31 * 640 * 2.0 ** -64
    kw = dict(eps=1e-5, adjacent=adjacent)
    out = ssd.ssd_qk_norm_rope(q, None, None, None, f, pos, **kw)[0].double().cpu().numpy()
    ref, err = om.norm_rope(q, None, f, pos, **kw)
    size = om._pair_size(om.norm_rope(q, None, None, None, **kw)[0], R, adjacent)
    assert (np.abs(out - ref) <= err + ang * size + 2.0 ** -24 * np.abs(ref)).all()
    d = torch.randn((b, L, h, D), generator=g).to(DEV)
    got = ssd.ssd_qk_norm_rope_bwd(q, None, None, None, f, d, None, pos, **kw)["dq"].double().cpu().numpy()
    r = om.norm_rope_bwd(q, None, f, d, pos, **kw)
    size = om._pair_size(d.double().cpu().numpy(), R, adjacent)
    v = q.double().cpu().numpy()
    s = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-5)
    turned = ang * s * (size + np.abs(v) * s * s * (size * np.abs(v)).mean(-1, keepdims=True))
    assert (np.abs(got - r["dv"]) <= r["e_dv"] + turned + 2.0 ** -24 * np.abs(r["dv"])).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("L", [37, 20011])
def test_an_infinite_gradient_gives_an_infinite_weight_gradient(dtype, L):
    """dq_weight[j] sums the incoming gradients of element j times positive values: where
    one of them is infinite, or all are, the sum is infinite, also where a CTA's last
    round has lanes without a head.  The other elements are what they are without."""
    g = torch.Generator().manual_seed(L)
    q = (torch.rand((1, L, 5, 128), generator=g) + 0.5).to(dtype).to(DEV)
    d = torch.randn((1, L, 5, 128), generator=g).to(dtype).to(DEV)
    clean = ssd.ssd_qk_norm_rope_bwd(q, None, None, None, None, d, None)["dq_weight"]
    rest = [j for j in range(128) if j not in (9, 77)]
    for everywhere in (True, False):
        dirty = d.clone()
        dirty[:, :, :, 9] = float("inf") if everywhere else dirty[:, :, :, 9]
        dirty[:, L - 1, 4, 77] = float("-inf")
        got = ssd.ssd_qk_norm_rope_bwd(q, None, None, None, None, dirty, None)["dq_weight"]
        assert got[77] == float("-inf") and (not everywhere or got[9] == float("inf"))
        assert torch.equal(got[rest], clean[rest])
