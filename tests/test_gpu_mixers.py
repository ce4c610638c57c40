"""The gated linear recurrence, the head norm with the position rotation and the
convolution's gradient on the GPU (through the C ABI), every element against the
fp64 definitions of oracle/mixers.py.

An element may differ by the definition's own fp32 error bound (its running
error, counted there) plus, where it is stored in fewer bits, half a step of that
type (finfo.eps / 2 of its value)."""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_b200 as ssd
from oracle import mixers as om

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def within(got, ref, err, what):
    half = torch.finfo(got.dtype).eps / 2
    g = got.detach().double().cpu().numpy()
    assert g.shape == ref.shape, what
    assert np.isfinite(g).all(), f"{what}: non-finite"
    # the rounded value lies within half a step of what fp32 had; a bf16 below the
    # normal range keeps an absolute step
    bound = err * (1 + half) + half * np.abs(ref) + torch.finfo(got.dtype).tiny
    bad = np.abs(g - ref) > bound
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(g - ref) / bound), g.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {g.size} elements; at {i} {g[i]} against "
                             f"{ref[i]}, bound {bound[i]:.3e}")


def dev(d):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


# ---- the gated linear recurrence --------------------------------------------
def scan_inputs(b, L, C, dtype, seed, resets=0, init=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)
    d = {"x": rn(b, L, C).to(dtype), "gate_a": rn(b, L, C).to(dtype), "gate_x": rn(b, L, C).to(dtype),
         "decay": torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(C, generator=g)) / 8.0))}
    d["init_state"] = rn(b, C) if init else None
    d["reset"] = (torch.rand((b, L), generator=g) < resets / L).to(torch.uint8) if resets else None
    return d, rn(b, L, C).to(dtype), rn(b, C) if init else None


SCAN = [
    # (b, L, C, dtype, resets, carried): one token, around the 64-token interval and
    # multiples of it, channels short of a tile and across several, restarts
    (1, 1, 8, BF, 0, True), (2, 2, 4, F32, 0, False), (3, 63, 24, BF, 0, True), (1, 64, 8, F32, 3, True),
    (2, 65, 72, BF, 4, False), (1, 127, 264, BF, 0, True), (2, 128, 64, F32, 0, False),
    (2, 129, 136, BF, 130, True), (4, 500, 40, F32, 9, True), (1, 1025, 200, BF, 5, True),
    (5, 1024, 128, BF, 0, False), (1, 2111, 12, F32, 2, True), (70, 33, 16, BF, 3, True),
    (2, 4099, 8, BF, 0, True),
]


@pytest.mark.parametrize("case", SCAN, ids=lambda c: "b{}_L{}_C{}_{}_r{}_{}".format(
    *c[:3], str(c[3]).split(".")[-1], c[4], "init" if c[5] else "zero"))
def test_gated_scan_and_gradient(case):
    b, L, C, dtype, resets, init = case
    d, dy, df = scan_inputs(b, L, C, dtype, seed=L * 7 + C, resets=resets, init=init)
    g = dev(d)
    y, fin, st = ssd.ssd_gated_scan(**g, return_final_state=True, return_states=True)
    ref = om.gated_scan(d["x"], d["gate_a"], d["gate_x"], d["decay"], d["init_state"], d["reset"])
    within(y, ref["y"], ref["e_y"], "y")
    within(fin, ref["final"], ref["e_final"], "final_state")
    within(st, ref["states"], ref["e_states"], "states")
    # the states and the final state are outputs of their own: y does not change without them
    assert torch.equal(y, ssd.ssd_gated_scan(**g))
    g.pop("init_state")
    o = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, d_final=None if df is None else df.to(DEV), **g)
    ref = om.gated_scan_bwd(d["x"], d["gate_a"], d["gate_x"], d["decay"], dy, d["init_state"], d["reset"], df)
    for k in ("dx", "dgate_a", "dgate_x", "ddecay", "d_init"):
        within(o[k], ref[k], ref["e_" + k], k)


@pytest.mark.parametrize("dtype,resets,scale,L", [(BF, 0, 0.25, 300), (BF, 6, 30.0, 700), (F32, 6, 30.0, 500),
                                                  (F32, 0, 2.5, 130), (BF, 200, 8.0, 333)])
def test_gated_scan_wide_decays(dtype, resets, scale, L):
    """Channels that keep everything beside channels that keep nothing, other
    scales, with and without restarts."""
    d, dy, df = scan_inputs(2, L, 72, dtype, seed=L, resets=resets)
    d["decay"] = torch.linspace(-9, 6, 72)[torch.randperm(72, generator=torch.Generator().manual_seed(1))]
    g = dict(dev(d), scale=scale)
    y, fin, st = ssd.ssd_gated_scan(**g, return_final_state=True, return_states=True)
    a = (d["x"], d["gate_a"], d["gate_x"], d["decay"])
    ref = om.gated_scan(*a, d["init_state"], d["reset"], scale=scale)
    within(y, ref["y"], ref["e_y"], "y")
    within(fin, ref["final"], ref["e_final"], "final_state")
    g.pop("init_state")
    o = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, d_final=df.to(DEV), **g)
    ref = om.gated_scan_bwd(*a, dy, d["init_state"], d["reset"], df, scale=scale)
    for k in ("dx", "dgate_a", "dgate_x", "ddecay", "d_init"):
        within(o[k], ref[k], ref["e_" + k], k)


def test_gated_scan_extreme_gates_and_decays():
    """Open and shut gates, decays of 1 and 0 and everything between, in both types."""
    vals = torch.tensor([-200.0, -30.0, -8.0, -1.0, 0.0, 1.0, 8.0, 30.0, 200.0])
    decs = torch.tensor([-120.0, -40.0, -12.0, -3.0, 0.0, 3.0, 20.0, 90.0])
    ga, gx = torch.meshgrid(vals, vals, indexing="ij")
    L = ga.numel()
    x = torch.linspace(-3, 3, L)[None, :, None].repeat(1, 1, 8)
    for dtype in (BF, F32):
        d = {"x": x.to(dtype), "gate_a": ga.reshape(1, L, 1).repeat(1, 1, 8).to(dtype).contiguous(),
             "gate_x": gx.reshape(1, L, 1).repeat(1, 1, 8).to(dtype).contiguous(), "decay": decs,
             "init_state": torch.full((1, 8), 2.0), "reset": None}
        g = dev(d)
        y, fin, st = ssd.ssd_gated_scan(**g, return_final_state=True, return_states=True)
        ref = om.gated_scan(d["x"], d["gate_a"], d["gate_x"], d["decay"], d["init_state"])
        # a gate at its end may be 2^-60 where it should be 0: e^-v is cut off there
        within(y, ref["y"], ref["e_y"] + 1e-15, "y")
        dy = torch.ones_like(d["x"])
        g.pop("init_state")
        o = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, **g)
        ref = om.gated_scan_bwd(d["x"], d["gate_a"], d["gate_x"], d["decay"], dy, d["init_state"])
        for k in ("dx", "dgate_a", "dgate_x", "ddecay", "d_init"):
            within(o[k], ref[k], ref["e_" + k] + 1e-13, k)


def test_gated_scan_restart_drops_infinities():
    """What one packed sequence overflowed to does not reach the next one, and a NaN
    stays in its own sequence and channel."""
    b, L, C = 2, 700, 16
    d, dy, _ = scan_inputs(b, L, C, BF, seed=5, init=True)
    clean = dict(d, reset=torch.zeros((b, L), dtype=torch.uint8))
    clean["reset"][:, [200, 450]] = 1
    dirty = {k: v.clone() for k, v in clean.items()}
    dirty["x"][0, 210, 3] = float("inf")
    dirty["gate_x"][1, 205, 5] = float("nan")
    dirty["init_state"][0, 7] = float("-inf")
    yc, sc = ssd.ssd_gated_scan(**dev(clean), return_states=True)
    yd, sd = ssd.ssd_gated_scan(**dev(dirty), return_states=True)
    assert torch.equal(yd[:, 450:], yc[:, 450:])
    # (h + em1 h of an infinite h is NaN: what overflowed stays visible, as one or the other)
    assert not torch.isfinite(yd[0, 210:450, 3]).any() and torch.isnan(yd[1, 205:450, 5]).all()
    assert not torch.isfinite(yd[0, :200, 7]).any() and torch.equal(yd[0, 200:, 7], yc[0, 200:, 7])
    for t in (clean, dirty):
        t.pop("init_state")
    dyd = dy.clone()
    dyd[0, 440, 9] = float("inf")   # the adjoint runs backwards from here, not past token 200
    gc = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=sc, **dev(clean))
    gd = ssd.ssd_gated_scan_bwd(dy=dyd.to(DEV), states=sd, **dev(dirty))
    for k in ("dx", "dgate_a", "dgate_x"):
        assert torch.equal(gd[k][:, 450:], gc[k][:, 450:]), k
        assert torch.equal(gd[k][0, :200, 9], gc[k][0, :200, 9]), k
        assert torch.equal(gd[k][0, 200:, 7], gc[k][0, 200:, 7]), k
    ok = [c for c in range(C) if c not in (3, 5, 7, 9)]
    assert torch.equal(gd["ddecay"][ok], gc["ddecay"][ok])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", [-60.0, -100.0, -3e38, float("-inf"), float("inf"), float("nan")])
def test_gated_scan_restart_does_not_use_its_decay_gate(dtype, gate):
    """A restarting token is i x whatever its gate_a (a padded or masked place may
    hold anything there): bitwise what a gate of 0 gives, in the scan, its gradient
    and the decode step; and that against the definition."""
    b, L, C = 2, 200, 24
    d, dy, df = scan_inputs(b, L, C, dtype, seed=11, init=True)
    d["reset"] = torch.zeros((b, L), dtype=torch.uint8)
    d["reset"][:, [0, 63, 64, 130, 199]] = 1
    runs = []
    for v in (0.0, gate):
        d["gate_a"][d["reset"] != 0] = v
        g = dev(d)
        y, fin, st = ssd.ssd_gated_scan(**g, return_final_state=True, return_states=True)
        h0 = g.pop("init_state")
        o = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, d_final=df.to(DEV), **g)
        new = torch.empty_like(h0)
        step = ssd.ssd_gated_state_update(h0, *(g[k][:, 64].contiguous() for k in ("x", "gate_a", "gate_x")),
                                          g["decay"], g["reset"][:, 64].contiguous(), new_state=new)
        runs.append({"y": y, "final": fin, "states": st, "step": step, "new": new, **o})
        if v == 0.0:
            ref = om.gated_scan(d["x"], d["gate_a"], d["gate_x"], d["decay"], d["init_state"], d["reset"])
            within(y, ref["y"], ref["e_y"], "y")
    for k in runs[0]:
        assert torch.equal(runs[0][k], runs[1][k]), k
    assert (runs[1]["dgate_a"][:, [0, 63, 64, 130, 199]] == 0).all()


def test_gated_scan_split_decode_and_bool_reset():
    """Resuming from the final state and stepping token by token give the scan's
    states, each within both bounds."""
    b, L, C = 3, 150, 40
    d, _, _ = scan_inputs(b, L, C, F32, seed=9, resets=3)
    g = dev(d)
    y, fin = ssd.ssd_gated_scan(**g, return_final_state=True)
    yb = ssd.ssd_gated_scan(**dict(g, reset=g["reset"].bool()))
    assert torch.equal(y, yb)
    cut = lambda a, z: {k: (v[:, a:z].contiguous() if k in ("x", "gate_a", "gate_x", "reset") else v)
                        for k, v in g.items()}
    y1, f1 = ssd.ssd_gated_scan(**cut(0, 77), return_final_state=True)
    y2, f2 = ssd.ssd_gated_scan(**dict(cut(77, L), init_state=f1), return_final_state=True)
    ref = om.gated_scan(*(d[k] for k in ("x", "gate_a", "gate_x", "decay", "init_state", "reset")))
    within(torch.cat([y1, y2], 1), ref["y"], ref["e_y"], "resumed y")
    within(f2, ref["final"], ref["e_final"], "resumed final state")
    state = g["init_state"].clone()
    for t in range(L):
        kept = state.clone()
        args = [g[k][:, t].contiguous() for k in ("x", "gate_a", "gate_x")]
        rs = g["reset"][:, t].contiguous()
        spare = torch.empty_like(state)
        y0 = ssd.ssd_gated_state_update(state, *args, g["decay"], rs, new_state=spare)
        assert torch.equal(state, kept)
        yt = ssd.ssd_gated_state_update(state, *args, g["decay"], rs)
        assert torch.equal(state, spare) and torch.equal(y0, yt)
        within(yt, ref["y"][:, t], ref["e_y"][:, t], f"decode step {t}")
    within(state, ref["final"], ref["e_final"], "decoded state")


@pytest.mark.parametrize("b,C,dtype,reset", [(1, 4, F32, False), (1, 8, BF, True), (3, 264, BF, True),
                                             (300, 520, BF, False), (17, 1540, F32, True), (513, 2048, BF, True)])
def test_gated_state_update(b, C, dtype, reset):
    d, _, _ = scan_inputs(b, 1, C, dtype, seed=b + C)
    one = {k: d[k][:, 0].contiguous() for k in ("x", "gate_a", "gate_x")}
    rs = torch.zeros(b, dtype=torch.uint8)
    rs[::2] = 1
    st = d["init_state"].to(DEV)
    if reset:
        st[0] = float("inf")  # a restarted row's old state is dropped, whatever it is
    y = ssd.ssd_gated_state_update(st, *(v.to(DEV) for v in one.values()), d["decay"].to(DEV),
                                   rs.to(DEV) if reset else None)
    ref, err = om.gated_state_update(d["init_state"], *one.values(), d["decay"], rs if reset else None)
    within(st, ref, err, "state")
    within(y, ref, err, "y")


def test_gated_scan_long_sequence():
    """A long sequence over many tiles: the definition on the channels 0 and C - 1."""
    b, L, C = 1, 30011, 520
    d, dy, df = scan_inputs(b, L, C, BF, seed=1, resets=2)
    g = dev(d)
    y, fin, st = ssd.ssd_gated_scan(**g, return_final_state=True, return_states=True)
    g.pop("init_state")
    o = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, d_final=df.to(DEV), **g)
    ch = [0, 263, C - 1]
    pick = lambda t: None if t is None else t[..., ch]
    a = [pick(d[k]) for k in ("x", "gate_a", "gate_x", "decay")]
    ref = om.gated_scan(*a, pick(d["init_state"]), d["reset"])
    within(pick(y), ref["y"], ref["e_y"], "y")
    within(pick(fin), ref["final"], ref["e_final"], "final")
    within(pick(st), ref["states"], ref["e_states"], "states")
    ref = om.gated_scan_bwd(*a, pick(dy), pick(d["init_state"]), d["reset"], pick(df))
    for k in ("dx", "dgate_a", "dgate_x", "ddecay", "d_init"):
        within(pick(o[k]), ref[k], ref["e_" + k], k)


def test_offsets_past_32_bits():
    """More than 2^31 elements in one tensor: the last batch row of each operator
    equals the same row computed alone."""
    b, L, C = 9, 65536, 4096  # 2.4 G elements
    gen = torch.Generator(device=DEV).manual_seed(0)
    big = torch.empty((b, L, C), dtype=BF, device=DEV)
    for i in range(b):
        big[i] = torch.randn((L, C), generator=gen, device=DEV)
    one = big[-1:].clone()
    dec = torch.full((C,), -3.0, device=DEV)
    y, st = ssd.ssd_gated_scan(big, big, big, dec, return_states=True)
    y1, st1 = ssd.ssd_gated_scan(one, one, one, dec, return_states=True)
    tol = 2.0 ** -7  # two bf16 roundings of values that differ by fp32 association
    assert torch.allclose(y[-1:].float(), y1.float(), rtol=tol, atol=1e-4)
    o = ssd.ssd_gated_scan_bwd(big, big, big, dec, big, st)
    o1 = ssd.ssd_gated_scan_bwd(one, one, one, dec, one, st1)
    for k in ("dx", "dgate_a", "dgate_x"):
        assert torch.allclose(o[k][-1:].float(), o1[k].float(), rtol=tol, atol=1e-4), k
    del o, o1, y, y1, st, st1
    q = big.view(b, L, 32, 128)
    f = 10000.0 ** (-torch.arange(64, device=DEV) / 64)
    qo, _ = ssd.ssd_qk_norm_rope(q, None, None, None, f)
    q1, _ = ssd.ssd_qk_norm_rope(one.view(1, L, 32, 128), None, None, None, f)
    assert torch.equal(qo[-1:], q1)
    del q1
    g = ssd.ssd_qk_norm_rope_bwd(q, None, None, None, f, qo, None)
    g1 = ssd.ssd_qk_norm_rope_bwd(one.view(1, L, 32, 128), None, None, None, f, qo[-1:], None)
    assert torch.equal(g["dq"][-1:], g1["dq"])
    del g, g1, qo
    w = torch.randn((C, 4), generator=gen, device=DEV)
    c = ssd.ssd_causal_conv1d_bwd(big, w, big)
    c1 = ssd.ssd_causal_conv1d_bwd(one, w, one)
    assert torch.allclose(c["dx"][-1:].float(), c1["dx"].float(), rtol=tol, atol=1e-4)


# ---- the head norm with the rotation ----------------------------------------
ROPE = [
    # (b, L, hq, hk, D, R, dtype, adjacent, lead, positions)
    (1, 1, 1, 1, 8, 0, BF, False, 0, None), (1, 1, 1, 1, 16, 16, BF, False, 0, "far"),
    (2, 3, 4, 2, 64, 64, BF, False, 0, None), (1, 37, 8, 8, 128, 128, BF, False, 64, None),
    (3, 5, 5, 1, 80, 80, BF, False, 0, "far"), (2, 9, 3, 1, 96, 48, BF, True, 8, "far"),
    (2, 11, 2, 2, 256, 256, BF, False, 0, None), (1, 65, 16, 2, 32, 16, BF, False, 0, "far"),
    (2, 7, 6, 3, 256, 64, F32, True, 4, "far"), (1, 130, 2, 1, 128, 128, F32, False, 0, "far"),
    (2, 3, 33, 0, 64, 32, F32, False, 0, None), (1, 2, 1, 65, 40, 32, BF, True, 0, "far"),
    (7, 301, 4, 1, 64, 64, BF, True, 16, None), (3, 1, 40, 8, 128, 112, F32, False, 0, "far"),
    (1, 9, 3, 2, 24, 16, F32, False, 0, "far"), (2, 3, 2, 2, 256, 0, F32, False, 0, None),
]


def rope_inputs(case, seed=0):
    b, L, hq, hk, D, R, dtype, adjacent, lead, positions = case
    g = torch.Generator().manual_seed(seed + b * L + D)
    buf = torch.randn((b, L, lead + (hq + hk) * D), generator=g).to(dtype).to(DEV)
    k = buf[..., lead:lead + hk * D].unflatten(-1, (hk, D)) if hk else None
    q = buf[..., lead + hk * D:].unflatten(-1, (hq, D))
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(DEV) for _ in range(2)]
    f = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(DEV) if R else None
    pos = torch.randint(0, 1 << 31, (b, L), generator=g).to(DEV) if positions else None
    d = [torch.randn((b, L, h, D), generator=g).to(dtype).to(DEV) for h in (hq, hk)]
    return buf, q, k, w, f, pos, d


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "b{}_L{}_q{}_k{}_D{}_R{}_{}_{}_lead{}_{}".format(
    *c[:6], str(c[6]).split(".")[-1], "adj" if c[7] else "half", c[8], c[9]))
def test_norm_rope_and_gradient(case):
    b, L, hq, hk, D, R, dtype, adjacent, lead, positions = case
    buf, q, k, w, f, pos, d = rope_inputs(case)
    before = buf.clone()
    kw = dict(eps=1e-5, adjacent=adjacent)
    qo, ko = ssd.ssd_qk_norm_rope(q, k, w[0], w[1], f, pos, **kw)
    o = ssd.ssd_qk_norm_rope_bwd(q, k, w[0], w[1], f, d[0], d[1] if hk else None, pos, **kw)
    assert torch.equal(buf, before)
    for name, v, wt, out, dout in (("q", q, w[0], qo, d[0]), ("k", k, w[1], ko, d[1])):
        if v is None:
            assert out is None and "dk" not in o
            continue
        ref, err = om.norm_rope(v, wt, f, pos, **kw)
        within(out, ref, err, name + "_out")
        ref = om.norm_rope_bwd(v, wt, f, dout, pos, **kw)
        within(o["d" + name], ref["dv"], ref["e_dv"], "d" + name)
        within(o[f"d{name}_weight"], ref["dweight"], ref["e_dweight"], f"d{name}_weight")
    # in place, inside the packed rows: the same values, and nothing else moves
    ssd.ssd_qk_norm_rope(q, k, w[0], w[1], f, pos, q_out=q, k_out=k, **kw)
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
    assert torch.equal(buf[..., :lead], before[..., :lead])
    # gradients written into slices of a packed row, given as slices of another
    gin = torch.cat([t.flatten(2) for t in (d[1], d[0])], -1)
    gout = torch.full_like(before, 7.0)
    dk = gout[..., lead:lead + hk * D].unflatten(-1, (hk, D)) if hk else None
    dq = gout[..., lead + hk * D:].unflatten(-1, (hq, D))
    q2 = before[..., lead + hk * D:].unflatten(-1, (hq, D))
    k2 = before[..., lead:lead + hk * D].unflatten(-1, (hk, D)) if hk else None
    o2 = ssd.ssd_qk_norm_rope_bwd(q2, k2, w[0], w[1], f, gin[..., hk * D:].unflatten(-1, (hq, D)),
                                  gin[..., :hk * D].unflatten(-1, (hk, D)) if hk else None, pos,
                                  out={"dq": dq, "dk": dk} if hk else {"dq": dq}, **kw)
    for name in o:
        assert torch.equal(o[name], o2[name]), name
    assert (gout[..., :lead] == 7.0).all()


def test_norm_rope_without_weights_and_zero_heads():
    case = (2, 5, 3, 2, 64, 64, F32, False, 0, None)
    _, q, k, w, f, pos, d = rope_inputs(case)
    one = torch.ones(64, device=DEV)
    a = ssd.ssd_qk_norm_rope(q, k, None, None, f)
    b = ssd.ssd_qk_norm_rope(q, k, one, one, f)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = ssd.ssd_qk_norm_rope_bwd(q, k, None, None, f, d[0], d[1])
    gb = ssd.ssd_qk_norm_rope_bwd(q, k, one, one, f, d[0], d[1])
    assert all(torch.equal(ga[n], gb[n]) for n in ga)
    # a head of zeros (padding) gives zeros, and a finite gradient: dv = w e / sqrt(eps)
    z = torch.zeros((1, 1, 1, 64), device=DEV)
    out, _ = ssd.ssd_qk_norm_rope(z, None, None, None, f)
    assert (out == 0).all()
    e = torch.ones_like(z)
    g = ssd.ssd_qk_norm_rope_bwd(z, None, None, None, f, e, None)
    assert torch.allclose(g["dq"], e / (1e-5 ** 0.5), rtol=1e-6) and (g["dq_weight"] == 0).all()


def test_norm_rope_negative_and_repeated_positions_and_high_frequencies():
    """Positions below zero, the same one twice, and more than a turn per position.
    The turns per position are off by up to 2^-53 of themselves (fp64) and 2^-65
    (the fraction), the angle in turns by that times |position|."""
    b, L, h, D, R = 1, 8, 2, 64, 32
    g = torch.Generator().manual_seed(3)
    q = torch.randn((b, L, h, D), generator=g).to(DEV)
    f = (torch.linspace(-7.5, 7.5, R // 2)).to(DEV)
    pos = torch.tensor([[-1, -70000, 5, 5, 0, -(1 << 20), 1 << 20, 3]]).to(DEV)
    turns = f.double().abs().max().item() / 6.28 * (1 << 20) * 2.0 ** -53 + (1 << 20) * 2.0 ** -65
    out, _ = ssd.ssd_qk_norm_rope(q, None, None, None, f, pos)
    ref, err = om.norm_rope(q, None, f, pos, eps=1e-5, adjacent=False)
    size = np.abs(om.norm_rope(q, None, None, None, eps=1e-5, adjacent=False)[0]).max()
    within(out, ref, err + 6.3 * turns * 2 * size, "out")
    assert torch.equal(ssd.ssd_qk_norm_rope(q[:, 2:4], None, None, None, f, pos[:, 2:4].contiguous())[0],
                       out[:, 2:4])


def test_norm_rope_nan_stays_in_its_head():
    q = torch.randn((2, 33, 5, 128), generator=torch.Generator().manual_seed(9)).to(BF).to(DEV)
    f = (10000.0 ** (-torch.arange(0, 128, 2) / 128)).to(DEV)
    dirty = q.clone()
    dirty[1, 7, 3, 100] = float("nan")
    dirty[0, 20, 0, 0] = float("inf")
    keep = torch.ones((2, 33, 5), dtype=torch.bool, device=DEV)
    keep[1, 7, 3] = keep[0, 20, 0] = False
    a, b = (ssd.ssd_qk_norm_rope(t, None, None, None, f)[0] for t in (q, dirty))
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[1, 7, 3]).all()
    e = torch.randn_like(q)
    a, b = (ssd.ssd_qk_norm_rope_bwd(t, None, None, None, f, e, None)["dq"] for t in (q, dirty))
    assert torch.equal(a[keep], b[keep])


# ---- the convolution's gradient ---------------------------------------------
CONV = [
    # (b, L, C, K, dtype, activation, carried)
    (1, 1, 8, 4, BF, True, True), (2, 2, 4, 8, F32, True, True), (1, 3, 16, 4, BF, False, False),
    (3, 31, 24, 3, F32, True, False), (2, 32, 72, 4, BF, True, True), (2, 33, 64, 5, BF, True, True),
    (1, 257, 136, 4, BF, True, False), (2, 500, 260, 3, F32, False, True), (1, 1030, 64, 2, BF, True, True),
    (4, 129, 40, 1, F32, True, False), (2, 300, 128, 6, BF, True, True), (1, 700, 200, 7, BF, False, True),
    (65, 40, 16, 4, BF, True, True), (1, 2500, 8, 4, F32, True, True), (2, 6, 264, 8, BF, True, True),
]


@pytest.mark.parametrize("case", CONV, ids=lambda c: "b{}_L{}_C{}_K{}_{}_{}_{}".format(
    *c[:4], str(c[4]).split(".")[-1], "silu" if c[5] else "linear", "init" if c[6] else "zero"))
def test_conv1d_bwd(case):
    b, L, C, K, dtype, act, init = case
    g = torch.Generator().manual_seed(L + C * K)
    rn = lambda *s: torch.randn(s, generator=g)
    x, dy = rn(b, L, C).to(dtype), rn(b, L, C).to(dtype)
    w, bias = rn(C, K) / K ** 0.5, rn(C)
    st, df = (rn(b, C, K - 1), rn(b, C, K - 1)) if init else (None, None)
    to = lambda t: None if t is None else t.to(DEV)
    o = ssd.ssd_causal_conv1d_bwd(to(x), to(w), to(dy), to(bias), to(st), to(df), activation=act)
    ref = om.conv1d_bwd(x, w, dy, bias, st, df, act)
    for k in ("dx", "dweight", "dbias") + (("d_init",) if K > 1 else ()):
        within(o[k], ref[k], ref["e_" + k], k)
    # no bias: the sum is taken without it
    o = ssd.ssd_causal_conv1d_bwd(to(x), to(w), to(dy), None, to(st), to(df), activation=act)
    ref = om.conv1d_bwd(x, w, dy, None, st, df, act)
    within(o["dx"], ref["dx"], ref["e_dx"], "dx without bias")


def test_conv1d_bwd_far_from_zero():
    """SiLU's gradient where e^-o leaves the fp32 range."""
    x = torch.linspace(-300, 300, 512)[None, :, None].repeat(1, 1, 4)
    w = torch.ones(4, 1)
    dy = torch.ones_like(x)
    o = ssd.ssd_causal_conv1d_bwd(x.to(DEV), w.to(DEV), dy.to(DEV))
    ref = om.conv1d_bwd(x, w, dy)
    within(o["dx"], ref["dx"], ref["e_dx"] + 1e-30, "dx")


# ---- together, and how calls are made ---------------------------------------
def test_a_trained_layer_end_to_end():
    """conv1d -> norm and rotation of C and B inside the packed rows -> ssd_fwd, and
    back through all three, against torch's reverse mode in fp64.  fp32; three
    stages, each within the library's 1e-4 rule."""
    b, L, H, P, N, G, K = 2, 192, 4, 64, 64, 2, 4
    X = H * P
    Cn = X + 2 * G * N
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(s, generator=g)
    u, w, bias = rn(b, L, Cn), rn(Cn, K) / 2, 0.1 * rn(Cn)
    dt, A, D = rn(b, L, H) - 2, -torch.rand(H, generator=g) - 0.5, rn(H)
    wc, wb = 1 + 0.1 * rn(N), 1 + 0.1 * rn(N)
    f = (100.0 ** (-torch.arange(0, N, 2, dtype=torch.float64) / N)).float()
    dy = rn(b, L, H, P)
    c = lambda t: t.to(DEV)
    xbc = ssd.ssd_causal_conv1d(c(u), c(w), c(bias))
    sl = lambda t: (t[..., :X].unflatten(-1, (H, P)), t[..., X:X + G * N].unflatten(-1, (G, N)),
                    t[..., X + G * N:].unflatten(-1, (G, N)))
    xs, B, C = sl(xbc)
    Cr, Br = ssd.ssd_qk_norm_rope(C, B, c(wc), c(wb), c(f))
    xs = xs.contiguous()
    y = ssd.ssd_fwd(xs, c(dt), c(A), Br, Cr, c(D), chunk=64)
    gs = ssd.ssd_bwd(xs, c(dt), c(A), Br, Cr, c(dy), c(D), chunk=64)
    dxbc = torch.empty_like(xbc)
    dxs, dB, dC = sl(dxbc)
    dxs.copy_(gs["dx"])
    gr = ssd.ssd_qk_norm_rope_bwd(C, B, c(wc), c(wb), c(f), gs["dC"], gs["dB"], out={"dq": dC, "dk": dB})
    gc = ssd.ssd_causal_conv1d_bwd(c(u), c(w), dxbc, c(bias))

    # the same layer in fp64, the scan as its masked product over token pairs
    t = {k: v.double().requires_grad_() for k, v in dict(u=u, w=w, bias=bias, wc=wc, wb=wb).items()}
    pre = torch.nn.functional.conv1d(torch.nn.functional.pad(t["u"].transpose(1, 2), (K - 1, 0)),
                                     t["w"][:, None], t["bias"], groups=Cn).transpose(1, 2)
    xs, B, C = sl(torch.nn.functional.silu(pre))

    def turn(v, wt):
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * wt
        ang = (torch.arange(L, dtype=torch.float64)[:, None] * f.double())[None, :, None]
        z = torch.complex(v[..., :N // 2], v[..., N // 2:]) * torch.polar(torch.ones_like(ang), ang)
        return torch.cat([z.real, z.imag], -1)
    C, B = turn(C, t["wc"]), turn(B, t["wb"])
    step = torch.nn.functional.softplus(dt.double())
    cum = torch.cumsum(step * A.double(), 1)
    seg = (cum[:, :, None] - cum[:, None]).masked_fill(~torch.ones(L, L).tril().bool()[None, :, :, None], -torch.inf)
    cb = torch.einsum("blgn,bsgn->blsg", C, B).repeat_interleave(H // G, -1)
    yr = torch.einsum("blsh,bsh,bshp->blhp", torch.exp(seg) * cb, step, xs) + D.double()[:, None] * xs
    (yr * dy.double()).sum().backward()
    for name, got, ref in (("y", y, yr.detach()), ("du", gc["dx"], t["u"].grad), ("dw", gc["dweight"], t["w"].grad),
                           ("dbias", gc["dbias"], t["bias"].grad), ("dwc", gr["dq_weight"], t["wc"].grad),
                           ("dwb", gr["dk_weight"], t["wb"].grad)):
        got, ref = got.double().cpu(), ref
        lim = 3e-4 * (ref.abs() + ref.pow(2).mean().sqrt())
        assert ((got - ref).abs() <= lim).all(), f"{name}: {((got - ref).abs() / lim).max():.2f} of the bound"


def test_conv_then_gated_scan_end_to_end():
    """conv1d -> gated recurrence and back, fp32, against torch's reverse mode in fp64
    (two stages of the library's 1e-4 rule)."""
    b, L, C, K = 2, 130, 24, 4
    d, dy, df = scan_inputs(b, L, C, F32, seed=3, resets=3)
    g = torch.Generator().manual_seed(8)
    u, w, bias = (torch.randn(s, generator=g) for s in ((b, L, C), (C, K), (C,)))
    c = lambda t: t.to(DEV)
    x = ssd.ssd_causal_conv1d(c(u), c(w), c(bias))
    rest = [c(d[k]) for k in ("gate_a", "gate_x", "decay")]
    y, st = ssd.ssd_gated_scan(x, *rest, c(d["init_state"]), c(d["reset"]), return_states=True)
    gs = ssd.ssd_gated_scan_bwd(x, *rest, c(dy), st, c(d["reset"]), c(df))
    gc = ssd.ssd_causal_conv1d_bwd(c(u), c(w), gs["dx"], c(bias))
    t = {k: v.double().requires_grad_() for k, v in dict(u=u, w=w, bias=bias, ga=d["gate_a"], gx=d["gate_x"],
                                                        dec=d["decay"], h0=d["init_state"]).items()}
    xr = torch.nn.functional.silu(torch.nn.functional.conv1d(
        torch.nn.functional.pad(t["u"].transpose(1, 2), (K - 1, 0)), t["w"][:, None], t["bias"],
        groups=C).transpose(1, 2))
    a = torch.exp(-8 * torch.nn.functional.softplus(t["dec"]) * torch.sigmoid(t["ga"])) \
        * (1 - d["reset"].double())[..., None]
    n = torch.sqrt(1 - a * a) * torch.sigmoid(t["gx"]) * xr
    h, ys = t["h0"], []
    for i in range(L):
        h = a[:, i] * h + n[:, i]
        ys.append(h)
    ((torch.stack(ys, 1) * dy.double()).sum() + (h * df.double()).sum()).backward()
    for name, got, ref in (("y", y, torch.stack(ys, 1).detach()), ("du", gc["dx"], t["u"].grad),
                           ("dw", gc["dweight"], t["w"].grad), ("dbias", gc["dbias"], t["bias"].grad),
                           ("dga", gs["dgate_a"], t["ga"].grad), ("dgx", gs["dgate_x"], t["gx"].grad),
                           ("ddecay", gs["ddecay"], t["dec"].grad), ("d_init", gs["d_init"], t["h0"].grad)):
        lim = 2e-4 * (ref.abs() + ref.pow(2).mean().sqrt())
        err = (got.double().cpu() - ref).abs()
        assert (err <= lim).all(), f"{name}: {(err / lim).max():.2f} of the bound"


def _calls(seed, dtype=BF):
    """One call of each operator on inputs of its own, as functions that return the
    output tensors (given buffers, so that they can be captured)."""
    d, dy, df = scan_inputs(2, 333, 72, dtype, seed, resets=3)
    g = dev(d)
    gb = {k: v for k, v in g.items() if k != "init_state"}
    case = (2, 37, 4, 2, 64, 64, dtype, False, 0, "far")
    _, q, k, w, f, pos, dq = rope_inputs(case, seed)
    gen = torch.Generator().manual_seed(seed)
    cw = torch.randn((72, 4), generator=gen).to(DEV)
    dyd = dy.to(DEV)
    st0 = torch.randn((5, 72), generator=gen).to(DEV)
    tok = [g[n][0, :5].contiguous() for n in ("x", "gate_a", "gate_x")]

    def scan():
        return list(ssd.ssd_gated_scan(**g, return_final_state=True, return_states=True))
    states = scan()[2]

    def scan_bwd():
        return list(ssd.ssd_gated_scan_bwd(dy=dyd, states=states, d_final=None,
                                           **gb).values())

    def update():
        new = torch.empty_like(st0)
        return [ssd.ssd_gated_state_update(st0, *tok, g["decay"], new_state=new), new]

    def rope():
        return list(ssd.ssd_qk_norm_rope(q, k, w[0], w[1], f, pos))

    def rope_bwd():
        return list(ssd.ssd_qk_norm_rope_bwd(q, k, w[0], w[1], f, dq[0], dq[1], pos).values())

    def conv_bwd():
        return list(ssd.ssd_causal_conv1d_bwd(g["x"], cw, dyd).values())
    return [scan, scan_bwd, update, rope, rope_bwd, conv_bwd]


@pytest.mark.parametrize("which", range(6), ids=["scan", "scan_bwd", "update", "rope", "rope_bwd", "conv_bwd"])
def test_repeated_streamed_and_captured_calls(which):
    """Bitwise the same: again, on another stream while the first runs too, and
    replayed from a graph, twice, with new inputs in between."""
    fn, other = _calls(1)[which], _calls(2)[which]
    want, want2 = fn(), other()
    torch.cuda.synchronize()
    for a, b in zip(want, fn()):
        assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):  # two calls at once
        with torch.cuda.stream(s1):
            outs.append((fn(), want))
        with torch.cuda.stream(s2):
            outs.append((other(), want2))
    torch.cuda.synchronize()
    for got, ref in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs = []
    for f in (fn, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for _ in range(2):
        for (g, out), ref in zip(graphs, (want, want2)):
            for t in out:
                t.fill_(0)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_stream_argument():
    s = torch.cuda.Stream()
    d, dy, _ = scan_inputs(1, 70, 8, BF, 3)
    g = dev(d)
    y, st = ssd.ssd_gated_scan(**g, return_states=True)
    torch.cuda.synchronize()
    y2, st2 = ssd.ssd_gated_scan(**g, return_states=True, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(st, st2)
    gb = {k: v for k, v in g.items() if k != "init_state"}
    a = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, **gb)
    torch.cuda.synchronize()
    b = ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, stream=s, **gb)
    s.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_nothing_outside_the_outputs_is_written():
    """Guard bands around every output and the workspace keep their fill."""
    b, L, C, K = 2, 77, 24, 4
    d, dy, df = scan_inputs(b, L, C, BF, 3)
    g = dev(d)
    bands = []

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        size = torch.finfo(dtype).bits // 8 if dtype.is_floating_point else 1
        buf = torch.full((512 + n * size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        t = buf[512:512 + n * size].view(dtype).view(shape)
        bands.append((buf, 512 + n * size))
        return t
    ns = -(-L // 64)
    y, fin, st = guarded((b, L, C), BF), guarded((b, C), F32), guarded((b, ns, C), F32)
    ssd.ssd_gated_scan(**g, y=y, final_state=fin, states=st)
    out = {"dx": guarded((b, L, C), BF), "dgate_a": guarded((b, L, C), BF), "dgate_x": guarded((b, L, C), BF),
           "ddecay": guarded((C,), F32), "d_init": guarded((b, C), F32)}
    gb = {k: v for k, v in g.items() if k != "init_state"}
    ws = guarded((ssd.ssd_gated_scan_bwd_workspace_size(b, L, C),), torch.uint8)
    ssd.ssd_gated_scan_bwd(dy=dy.to(DEV), states=st, out=out, workspace=ws, **gb)
    one = [g[k][:, 0].contiguous() for k in ("x", "gate_a", "gate_x")]
    ssd.ssd_gated_state_update(guarded((b, C), F32).zero_(), *one, g["decay"], y=guarded((b, C), BF))
    q = dy.to(DEV).view(b, L, 1, C)
    f = torch.ones(8, device=DEV)
    ssd.ssd_qk_norm_rope(q, q, None, None, f, q_out=guarded(q.shape, BF), k_out=guarded(q.shape, BF))
    ws = guarded((ssd.ssd_qk_norm_rope_bwd_workspace_size(b, L, 1, 1, C, 16),), torch.uint8)
    ssd.ssd_qk_norm_rope_bwd(q, q, None, None, f, q, q, workspace=ws, out={
        "dq": guarded(q.shape, BF), "dk": guarded(q.shape, BF), "dq_weight": guarded((C,), F32),
        "dk_weight": guarded((C,), F32)})
    w = torch.randn((C, K), device=DEV)
    ws = guarded((ssd.ssd_causal_conv1d_bwd_workspace_size(b, L, C, K),), torch.uint8)
    ssd.ssd_causal_conv1d_bwd(g["x"], w, dy.to(DEV), workspace=ws, out={
        "dx": guarded((b, L, C), BF), "dweight": guarded((C, K), F32), "dbias": guarded((C,), F32),
        "d_init": guarded((b, C, K - 1), F32)})
    torch.cuda.synchronize()
    for buf, end in bands:
        assert (buf[:512] == 0xA5).all() and (buf[end:] == 0xA5).all()


def test_largest_batches_and_head_counts():
    """The limits of the grid: the last batch row or head alone gives the same."""
    b = 65535
    g = torch.Generator(device=DEV).manual_seed(2)
    x, ga, gx, dy = (torch.randn((b, 2, 8), generator=g, device=DEV).to(BF) for _ in range(4))
    dec = torch.linspace(-6, 1, 8, device=DEV)
    one = [t[-1:].clone() for t in (x, ga, gx)]
    y, fin, st = ssd.ssd_gated_scan(x, ga, gx, dec, return_final_state=True, return_states=True)
    y1, fin1, st1 = ssd.ssd_gated_scan(*one, dec, return_final_state=True, return_states=True)
    assert torch.equal(y[-1:], y1) and torch.equal(fin[-1:], fin1)
    o = ssd.ssd_gated_scan_bwd(x, ga, gx, dec, dy, st)
    o1 = ssd.ssd_gated_scan_bwd(*one, dec, dy[-1:].clone(), st1)
    assert all(torch.equal(o[k][-1:], o1[k]) for k in ("dx", "dgate_a", "dgate_x", "d_init"))
    s, s1 = fin.clone(), fin[-1:].clone()
    y = ssd.ssd_gated_state_update(s, *(t[:, 0].contiguous() for t in (x, ga, gx)), dec)
    y1 = ssd.ssd_gated_state_update(s1, *(t[:, 0].contiguous() for t in one), dec)
    assert torch.equal(y[-1:], y1) and torch.equal(s[-1:], s1)
    w = torch.randn((8, 4), generator=g, device=DEV)
    c = ssd.ssd_causal_conv1d_bwd(x, w, dy)
    c1 = ssd.ssd_causal_conv1d_bwd(one[0], w, dy[-1:].clone())
    assert torch.equal(c["dx"][-1:], c1["dx"]) and torch.equal(c["d_init"][-1:], c1["d_init"])
    q = torch.randn((1, 2, 65535, 16), generator=g, device=DEV).to(BF)
    k = torch.randn((1, 2, 1, 16), generator=g, device=DEV).to(BF)
    f = torch.rand(8, generator=g, device=DEV)
    qo, ko = ssd.ssd_qk_norm_rope(q, k, None, None, f)
    q1, k1 = ssd.ssd_qk_norm_rope(q[:, :, -1:].contiguous(), k, None, None, f)
    assert torch.equal(qo[:, :, -1:], q1) and torch.equal(ko, k1)
    g2 = ssd.ssd_qk_norm_rope_bwd(q, k, None, None, f, qo, ko)
    g1 = ssd.ssd_qk_norm_rope_bwd(q[:, :, -1:].contiguous(), k, None, None, f, q1, k1)
    assert torch.equal(g2["dq"][:, :, -1:], g1["dq"]) and torch.equal(g2["dk"], g1["dk"])


def test_calls_from_several_threads():
    """Host threads with a stream each, at the same time."""
    import threading
    fns = [_calls(s) for s in (1, 2, 3, 4)]
    want = [[fn() for fn in row] for row in fns]
    torch.cuda.synchronize()
    bad = []

    def work(row, refs):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                outs = [fn() for fn in row]
                s.synchronize()
                bad.extend(i for i, (a, b) in enumerate(zip(outs, refs))
                           if not all(torch.equal(p, q) for p, q in zip(a, b)))
    threads = [threading.Thread(target=work, args=a) for a in zip(fns, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


FIRST_CALLS = r"""
import sys, torch
sys.path.insert(0, ROOT)
import mamba_ssd_scan_b200 as ssd
g = torch.Generator(device="cuda").manual_seed(0)
rn = lambda *s: torch.randn(s, generator=g, device="cuda")
x, ga, gx, dy = (rn(2, 300, 64).bfloat16() for _ in range(4))
dec, q, f, w = torch.full((64,), -4.0, device="cuda"), rn(2, 9, 4, 64).bfloat16(), rn(32), rn(64, 4)
st, s0 = torch.zeros(2, 5, 64, device="cuda"), torch.zeros(2, 64, device="cuda")
one = [t[:, 0].contiguous() for t in (x, ga, gx)]
for run in (lambda: [ssd.ssd_gated_scan(x, ga, gx, dec)],
            lambda: list(ssd.ssd_gated_scan_bwd(x, ga, gx, dec, dy, st).values()),
            lambda: [ssd.ssd_gated_state_update(s0, *one, dec, new_state=torch.empty_like(s0))],
            lambda: [ssd.ssd_qk_norm_rope(q, None, None, None, f)[0]],
            lambda: list(ssd.ssd_qk_norm_rope_bwd(q, None, None, None, f, q, None).values()),
            lambda: list(ssd.ssd_causal_conv1d_bwd(x, w, dy).values())):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    graph.replay()
    torch.cuda.synchronize()
    again = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, again))
print("CAPTURE-OK")
"""


def test_first_call_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"ROOT = {root!r}\n" + FIRST_CALLS], capture_output=True, text=True,
                       timeout=180)
    assert r.returncode == 0 and "CAPTURE-OK" in r.stdout, r.stdout + r.stderr
