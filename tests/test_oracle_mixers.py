"""The fp64 definitions the GPU tests of the gated recurrence, the head norm with
the rotation and the convolution's gradient compare with, pinned without their
own code: closed forms, differences, and torch's reverse mode on forms written
apart (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import mixers as om


def _inputs(b=2, L=9, C=3, seed=0):
    g = np.random.default_rng(seed)
    x, ga, gx, dy = (g.standard_normal((b, L, C)) for _ in range(4))
    decay = g.standard_normal(C) - 2.0
    init, df = g.standard_normal((b, C)), g.standard_normal((b, C))
    reset = np.zeros((b, L))
    reset[0, 4] = reset[1, 0] = 1
    return x, ga, gx, decay, dy, init, df, reset


def test_scan_closed_forms():
    x, ga, gx, decay, dy, init, df, reset = _inputs()
    # a decay gate that is shut (a = 1) keeps the state and takes nothing in
    f = om.gated_scan(x, np.full_like(ga, -1e9), gx, decay, init)
    assert np.allclose(f["y"], init[:, None], atol=0, rtol=1e-15)
    # a = 1/2 by hand: softplus(decay) = ln 2 at decay 0, sigma(0) = 1/2, scale 2
    f = om.gated_scan(np.ones((1, 3, 1)), np.zeros((1, 3, 1)), np.zeros((1, 3, 1)), np.zeros(1),
                      np.array([[4.0]]), scale=2.0)
    u = np.sqrt(0.75) / 2
    assert np.allclose(f["y"][0, :, 0], [2 + u, 1 + 1.5 * u, 0.5 + 1.75 * u], rtol=1e-15)
    # a restart forgets everything before it, an infinite state included
    init2 = init.copy()
    init2[1] = np.inf
    f = om.gated_scan(x, ga, gx, decay, init2, reset)
    tail = om.gated_scan(x[1:], ga[1:], gx[1:], decay, None, None)
    assert np.allclose(f["y"][1, 0], (om.sigma(gx) * x)[1, 0]) and np.isfinite(f["y"]).all()
    assert not np.allclose(f["y"][1, 0], tail["y"][0, 0])  # without the restart n < 1
    # split and resume
    whole = om.gated_scan(x, ga, gx, decay, init)
    a = om.gated_scan(x[:, :5], ga[:, :5], gx[:, :5], decay, init)
    c = om.gated_scan(x[:, 5:], ga[:, 5:], gx[:, 5:], decay, a["final"])
    assert np.allclose(np.concatenate([a["y"], c["y"]], 1), whole["y"], rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("use_reset", [False, True])
def test_scan_gradients_against_differences_and_autograd(use_reset):
    x, ga, gx, decay, dy, init, df, reset = _inputs()
    rs = reset if use_reset else None
    o = om.gated_scan_bwd(x, ga, gx, decay, dy, init, rs, df)
    ins = {"dx": x, "dgate_a": ga, "dgate_x": gx, "ddecay": decay, "d_init": init}

    def J():
        f = om.gated_scan(x, ga, gx, decay, init, rs)
        return (f["y"] * dy).sum() + (f["final"] * df).sum()
    for name, arr in ins.items():
        num = np.zeros_like(arr)
        for idx in np.ndindex(*arr.shape):
            keep = arr[idx]
            arr[idx] = keep + 1e-6
            up = J()
            arr[idx] = keep - 1e-6
            num[idx] = (up - J()) / 2e-6
            arr[idx] = keep
        assert np.allclose(o[name], num, rtol=1e-6, atol=1e-7), name
    # the unrolled double sum in torch: h_t = sum_s prod(a_{s+1..t}) n_s i_s x_s
    t = {k: torch.tensor(v, requires_grad=True) for k, v in ins.items()}
    on = torch.tensor(1 - reset if use_reset else np.ones_like(reset))[..., None]
    la = -8.0 * torch.nn.functional.softplus(t["ddecay"]) * torch.sigmoid(t["dgate_a"])
    a = torch.exp(la) * on
    u = torch.sqrt(1 - a * a) * torch.sigmoid(t["dgate_x"]) * t["dx"]
    ys = []
    for i in range(x.shape[1]):
        h = torch.prod(a[:, :i + 1], 1) * t["d_init"]
        for s in range(i + 1):
            h = h + torch.prod(a[:, s + 1:i + 1], 1) * u[:, s]
        ys.append(h)
    (sum((y * torch.tensor(dy[:, i])).sum() for i, y in enumerate(ys))
     + (ys[-1] * torch.tensor(df)).sum()).backward()
    for name in ins:
        assert np.allclose(o[name], t[name].grad.numpy(), rtol=1e-9, atol=1e-10), name


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_rope_properties_and_gradient(rot, adjacent):
    g = np.random.default_rng(3)
    v, d = g.standard_normal((2, 3, 2, 8)), g.standard_normal((2, 3, 2, 8))
    w = 1 + 0.1 * g.standard_normal(8)
    f = 10.0 ** -np.arange(rot // 2) if rot else None
    pos = np.array([[0, 7, 100000], [5, 6, 7]])
    out, _ = om.norm_rope(v, w, f, pos, adjacent=adjacent)
    # position 0 and the unrotated rest: the plain norm; a rotation keeps lengths
    plain = v / np.sqrt((v * v).mean(-1, keepdims=True) + 1e-5) * w
    assert np.allclose(out[0, 0], plain[0, 0], rtol=1e-14)
    assert np.allclose(out[..., rot:], plain[..., rot:], rtol=1e-14)
    assert np.allclose((out ** 2).sum(-1), (plain ** 2).sum(-1), rtol=1e-12)
    if rot:  # products of two rotated heads depend on the distance of their tokens only
        far, _ = om.norm_rope(v[1:], w, f, pos[1:] + 1000, adjacent=adjacent)
        assert np.allclose((far[0, 0] * far[0, 2]).sum(-1), (out[1, 0] * out[1, 2]).sum(-1), rtol=1e-9)
        # a quarter turn by hand: (a, b) -> (-b, a)
        q, _ = om.norm_rope(v, w, np.full(rot // 2, np.pi / 2), np.ones((2, 3), int), adjacent=adjacent)
        p0, p1 = (0, 1) if adjacent else (0, rot // 2)
        assert np.allclose(q[..., p0], -plain[..., p1]) and np.allclose(q[..., p1], plain[..., p0])
    o = om.norm_rope_bwd(v, w, f, d, pos, adjacent=adjacent)
    for name, arr in (("dv", v), ("dweight", w)):
        num = np.zeros_like(arr)
        for idx in np.ndindex(*arr.shape):
            keep = arr[idx]
            arr[idx] = keep + 1e-6
            up = (om.norm_rope(v, w, f, pos, adjacent=adjacent)[0] * d).sum()
            arr[idx] = keep - 1e-6
            num[idx] = (up - (om.norm_rope(v, w, f, pos, adjacent=adjacent)[0] * d).sum()) / 2e-6
            arr[idx] = keep
        assert np.allclose(o[name], num, rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("L,K,act", [(7, 4, True), (2, 5, True), (6, 1, False), (1, 3, False)])
def test_conv_gradient_against_the_oracle_and_torch(orc, L, K, act):
    g = np.random.default_rng(L * K)
    b, C = 2, 3
    x, dy = g.standard_normal((b, L, C)), g.standard_normal((b, L, C))
    w, bias = g.standard_normal((C, K)), g.standard_normal(C)
    init, df = g.standard_normal((b, C, K - 1)), g.standard_normal((b, C, K - 1))
    o = om.conv1d_bwd(x, w, dy, bias, init, df, act)
    t = [torch.tensor(v, requires_grad=True) for v in (x, w, bias, init)]
    xin = torch.cat([t[3], t[0].transpose(1, 2)], 2)
    y = torch.nn.functional.conv1d(xin, t[1][:, None], t[2], groups=C)
    y = torch.nn.functional.silu(y) if act else y
    y = y.transpose(1, 2)
    # the forward that is differentiated here is the library oracle's
    ref, fin = orc.causal_conv1d(x, w, bias, init, act)
    assert np.allclose(y.detach().numpy(), ref, rtol=1e-12, atol=1e-12)
    ((y * torch.tensor(dy)).sum() + (xin[:, :, L:] * torch.tensor(df)).sum()).backward()
    for name, v in zip(("dx", "dweight", "dbias", "d_init"), t):
        assert np.allclose(o[name], v.grad.numpy(), rtol=1e-10, atol=1e-12), name
