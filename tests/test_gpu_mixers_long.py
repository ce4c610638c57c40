"""The newer kernels' steady states against the fp64 definitions of oracle/mixers.py:
several tiles per CTA in the head norm, segments longer than the ring in the
convolution's gradient, four rows per thread in the decode step.  The sizes are
those at which 148 SMs run them; tests/test_mixers_long_host.py holds the launch
rules to that."""
import pytest
import torch

import mamba_ssd_scan_b200 as ssd
from oracle import mixers as om
from test_gpu_mixers import rope_inputs, scan_inputs, within

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

LONG_ROPE = [
    # several tiles per CTA, the last one ragged; forward and backward
    (1, 20011, 8, 8, 128, 128, BF, False, 64, None), (3, 20011, 5, 1, 64, 32, F32, True, 4, "far"),
    (2, 5003, 32, 8, 64, 64, BF, True, 0, "far"), (1, 20011, 3, 0, 256, 64, F32, False, 0, None),
]


@pytest.mark.parametrize("case", LONG_ROPE, ids=lambda c: "b{}_L{}_q{}_k{}_D{}_R{}_{}_{}".format(
    *c[:6], str(c[6]).split(".")[-1], "adj" if c[7] else "half"))
def test_norm_rope_over_several_tiles(case):
    b, L, hq, hk, D, R, dtype, adjacent, lead, positions = case
    buf, q, k, w, f, pos, d = rope_inputs(case)
    kw = dict(eps=1e-5, adjacent=adjacent)
    qo, ko = ssd.ssd_qk_norm_rope(q, k, w[0], w[1], f, pos, **kw)
    o = ssd.ssd_qk_norm_rope_bwd(q, k, w[0], w[1], f, d[0], d[1] if hk else None, pos, **kw)
    for name, v, wt, out, dout in (("q", q, w[0], qo, d[0]), ("k", k, w[1], ko, d[1])):
        if v is None:
            continue
        ref, err = om.norm_rope(v, wt, f, pos, **kw)
        within(out, ref, err, name + "_out")
        del ref, err
        ref = om.norm_rope_bwd(v, wt, f, dout, pos, **kw)
        within(o["d" + name], ref["dv"], ref["e_dv"], "d" + name)
        within(o[f"d{name}_weight"], ref["dweight"], ref["e_dweight"], f"d{name}_weight")


@pytest.mark.parametrize("b,L,C,K,dtype,act", [(8, 1500, 2304, 4, BF, True), (8, 1111, 2304, 8, BF, True),
                                               (8, 1501, 1536, 3, F32, False)])
def test_conv1d_bwd_long_segments(b, L, C, K, dtype, act):
    """dx, dweight, dbias and d_init of every 37th channel (each channel is a sum of its
    own) at segments of more batches than the ring holds."""
    g = torch.Generator().manual_seed(L)
    rn = lambda *s: torch.randn(s, generator=g)
    x, dy = rn(b, L, C).to(dtype), rn(b, L, C).to(dtype)
    w, bias = rn(C, K) / K ** 0.5, rn(C)
    st, df = rn(b, C, K - 1), rn(b, C, K - 1)
    o = ssd.ssd_causal_conv1d_bwd(*(t.to(DEV) for t in (x, w, dy, bias, st, df)), activation=act)
    ch = torch.cat([torch.arange(0, C, 37), torch.tensor([C - 1])])
    ref = om.conv1d_bwd(x[..., ch], w[ch], dy[..., ch], bias[ch], st[:, ch], df[:, ch], act)
    on = ch.to(DEV)
    for k, got in (("dx", o["dx"][..., on]), ("dweight", o["dweight"][on]), ("dbias", o["dbias"][on]),
                   ("d_init", o["d_init"][:, on])):
        within(got, ref[k], ref["e_" + k], k)


@pytest.mark.parametrize("b,C,dtype,reset", [(257, 5120, BF, True), (258, 5120, F32, True), (513, 2560, F32, False),
                                             (1027, 1544, BF, True)])
def test_gated_state_update_four_rows_per_thread(b, C, dtype, reset):
    d, _, _ = scan_inputs(b, 1, C, dtype, seed=b + C)
    one = {k: d[k][:, 0].contiguous() for k in ("x", "gate_a", "gate_x")}
    rs = torch.zeros(b, dtype=torch.uint8)
    rs[::3] = 1
    st = d["init_state"].to(DEV)
    if reset:
        st[0] = float("inf")  # a restarted row's old state is dropped, whatever it is
    new = torch.empty_like(st)
    args = [v.to(DEV) for v in one.values()] + [d["decay"].to(DEV), rs.to(DEV) if reset else None]
    kept = st.clone()
    y0 = ssd.ssd_gated_state_update(st, *args, new_state=new)
    assert torch.equal(st, kept)
    y = ssd.ssd_gated_state_update(st, *args)
    assert torch.equal(y, y0) and torch.equal(st, new)
    ref, err = om.gated_state_update(d["init_state"], *one.values(), d["decay"], rs if reset else None)
    within(st, ref, err, "state")
    within(y, ref, err, "y")
