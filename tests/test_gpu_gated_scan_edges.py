"""The gated linear recurrence where it could go wrong: states that are large beside
what a token keeps of them, and states that are not finite."""
import pytest
import torch

import mamba_ssd_scan_b200 as ssd
from oracle import mixers as om
from test_gpu_mixers import dev, within

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def wide_inputs(b, L, C, dtype, seed, resets=0):
    """Decays from 1 down to e^-48, inputs and incoming gradients of sizes from 1e-3 to
    1e6 behind gates from open to nearly shut (e^-10: their own rounding stays
    within the definition's bound), a carried state and a final gradient of 1e4 to
    1e8."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)
    sized = lambda lo, hi, *s: rn(*s) * 10 ** (lo + (hi - lo) * torch.rand(s, generator=g))
    d = {"x": sized(-3, 6, b, L, C).to(dtype), "gate_a": (1 + rn(b, L, C)).clamp(-3, 4).to(dtype),
         "gate_x": (14 * torch.rand((b, L, C), generator=g) - 10).to(dtype),
         "decay": torch.linspace(-6, 6, C)[torch.randperm(C, generator=g)],
         "init_state": sized(4, 8, b, C), "reset": None}
    if resets:
        d["reset"] = (torch.rand((b, L), generator=g) < resets / L).to(torch.uint8)
    return d, sized(-3, 6, b, L, C).to(dtype), sized(4, 8, b, C)


def check_scan(d, dy, df, what=""):
    g = dev(d)
    y, fin, st = ssd.ssd_gated_scan(**g, return_final_state=True, return_states=True)
    ref = om.gated_scan(d["x"], d["gate_a"], d["gate_x"], d["decay"], d["init_state"], d["reset"])
    within(y, ref["y"], ref["e_y"], what + "y")
    within(fin, ref["final"], ref["e_final"], what + "final_state")
    within(st, ref["states"], ref["e_states"], what + "states")
    g.pop("init_state")
    o = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, d_final=df.to(DEV), **g)
    ref = om.gated_scan_bwd(d["x"], d["gate_a"], d["gate_x"], d["decay"], dy, d["init_state"], d["reset"], df)
    for k in ("dx", "dgate_a", "dgate_x", "ddecay", "d_init"):
        within(o[k], ref[k], ref["e_" + k], what + k)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,L,C,resets", [(2, 1, 72, 0), (3, 9, 64, 0), (1, 70, 200, 4), (1, 1500, 72, 0),
                                          (2, 1301, 136, 40)])
def test_small_decays_keep_what_is_left(dtype, b, L, C, resets):
    """A token that keeps little of a large state keeps that little accurately: the
    definition's bound counts a |h|, not |h|."""
    check_scan(*wide_inputs(b, L, C, dtype, seed=L, resets=resets))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_decode_steps_at_small_decays(dtype):
    d, _, _ = wide_inputs(600, 12, 72, dtype, seed=4)
    g = dev(d)
    ref = om.gated_scan(d["x"], d["gate_a"], d["gate_x"], d["decay"], d["init_state"])
    st = g["init_state"].clone()
    for t in range(12):
        y = ssd.ssd_gated_state_update(st, *(g[k][:, t].contiguous() for k in ("x", "gate_a", "gate_x")), g["decay"])
        within(y, ref["y"][:, t], ref["e_y"][:, t], f"y of step {t}")
    within(st, ref["final"], ref["e_final"], "state")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("decay", [-6.0, 3.0])
def test_an_infinite_end_is_the_final_state(dtype, decay):
    """The final state is the last token's, infinite or not, and an infinite d_final
    enters at the last token, wherever the sequence ends in its group of tokens."""
    g = torch.Generator().manual_seed(0)
    C = 8
    for L in list(range(1, 18)) + [63, 64, 65, 500, 1029]:
        x, ga, gx, dy = (torch.randn((1, L, C), generator=g).to(dtype).to(DEV) for _ in range(4))
        x[0, L - 1, 2], x[0, L - 1, 5] = float("inf"), float("-inf")
        dec = torch.full((C,), decay, device=DEV)
        y, fin, st = ssd.ssd_gated_scan(x, ga, gx, dec, return_final_state=True, return_states=True)
        assert y[0, L - 1, 2] == float("inf") and y[0, L - 1, 5] == float("-inf")
        assert fin[0, 2] == float("inf") and fin[0, 5] == float("-inf"), L
        assert torch.isfinite(fin[0, [0, 1, 3, 4, 6, 7]]).all(), L
        x[0, L - 1, 2], x[0, L - 1, 5] = 1.0, 1.0
        df = torch.zeros((1, C), device=DEV)
        df[0, 3] = float("inf")
        o = ssd.ssd_gated_scan_bwd(x, ga, gx, dec, dy, st, d_final=df)
        # dx = g n i, g infinite
        assert torch.isinf(o["dx"][0, L - 1, 3]) and o["dx"][0, L - 1, 3] > 0, L
        assert torch.isfinite(o["dx"][0, :, [0, 1, 4, 6, 7]]).all(), L


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_nearly_shut_gates_relative_to_what_they_add(dtype):
    """Down to where a gate counts as shut a token adds sqrt(2 scale softplus(decay) r) i x
    with r as small as e^-86: outputs of 1e-18 and their gradients keep their relative
    accuracy.  A bf16 gate's e^-v is off by up to half an ulp of v log2 e in the
    exponent: 2^-19 ln 2 of itself from 2^5 on, 2^-18 ln 2 from 2^6 on; half of that in
    the square root."""
    ga = torch.arange(-86.0, -30.0, 4.0)
    L, C = ga.numel(), 8
    x = torch.linspace(1, 2, L)[None, :, None].repeat(1, 1, C).to(dtype)
    gx = torch.full((1, L, C), 6.0).to(dtype)
    gav = ga[None, :, None].repeat(1, 1, C).to(dtype)
    dec = torch.linspace(-3, 3, C)
    dy = torch.ones(1, L, C, dtype=dtype)
    # a token per call: the states before it would hide it
    for t in range(L):
        one = [v[:, t:t + 1].contiguous() for v in (x, gav, gx)]
        g = [v.to(DEV) for v in one] + [dec.to(DEV)]
        y, st = ssd.ssd_gated_scan(*g, return_states=True)
        ref = om.gated_scan(*one, dec)
        more = 2.0 ** -18 * 0.7 if dtype is BF else 0.0
        within(y, ref["y"], ref["e_y"] + more * abs(ref["y"]), f"y at gate {ga[t]}")
        o = ssd.ssd_gated_scan_bwd(*g, dy[:, t:t + 1].to(DEV), st)
        ref = om.gated_scan_bwd(*one, dec, dy[:, t:t + 1])
        for k in ("dx", "dgate_x"):
            within(o[k], ref[k], ref["e_" + k] + more * abs(ref[k]), f"{k} at gate {ga[t]}")
