"""fp64 definitions of the gated linear recurrence, the head norm with the
position rotation and the convolution's gradient, token by token in numpy (test
infrastructure; it shares no code with the CUDA path).

Each function returns the values and, beside them, a bound on what fp32
arithmetic may differ by: the first-order running error of the same formulas.
``U`` = 2^-24 is one fp32 rounding.  ``D`` = 16 U covers the chain behind one
gated coefficient (a product, e^x and a quotient per gate at 2 U each, the decay's
product and expm1, the square root); a recurrence step rounds its state
twice, and twice more where a state is composed from partial ones.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126  # fp32 results below it may be zero
D = 16 * U
INTERVAL = 64


def _np(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().to("cpu").double().numpy()
    return np.asarray(a, dtype=np.float64)


def sigma(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def gates(gate_a, gate_x, decay, scale, reset):
    """r, i, la, a, em1 = a - 1, n of every token; a = 0, n = 1 where reset."""
    r, i = sigma(gate_a), sigma(gate_x)
    la = -scale * softplus(decay) * r
    a, em1 = np.exp(la), np.expm1(la)
    if reset is not None:
        a = np.where((reset != 0)[..., None], 0.0, a)
        em1 = np.where((reset != 0)[..., None], -1.0, em1)
    n = np.sqrt(-em1 * (2.0 + em1))
    return r, i, la, a, em1, n


def kept(la, a, em1, h):
    """Error of a h: with a decay near 1 as h + em1 h, em1 off by D of itself, beyond as
    e^la h, la off by D of itself; the old state is never rounded at its own size
    where little of it is kept."""
    return np.where(la >= -0.25, np.abs(em1) * D, a * (1.0 + np.abs(la)) * D + TINY) * np.abs(h)


def gated_scan(x, gate_a, gate_x, decay, init=None, reset=None, scale=8.0):
    """[b, L, C] arrays -> dict of y, final, states and their error bounds e_*."""
    x, gate_a, gate_x, decay = map(_np, (x, gate_a, gate_x, decay))
    init, reset = _np(init), _np(reset)
    b, L, C = x.shape
    r, i, la, decays, em1, n = gates(gate_a, gate_x, decay, scale, reset)
    u = n * i * x
    h = np.zeros((b, C)) if init is None else init.copy()
    err = np.zeros((b, C))
    y, e_y = np.empty_like(x), np.empty_like(x)
    states, e_states = [], []
    for t in range(L):
        if t % INTERVAL == 0:
            states.append(h.copy())
            e_states.append(err.copy())
        a = decays[:, t]
        keep = a > 0  # a restart forgets the state and its error exactly
        if reset is not None:
            keep = keep & (reset[:, t] == 0)[:, None]
        hn = np.where(keep, a * np.where(keep, h, 0.0), 0.0) + u[:, t]
        # what is kept of the old state, then four roundings of the new one
        err = np.where(keep, a * err + kept(la[:, t], a, em1[:, t], np.where(keep, h, 0.0)), 0.0) \
            + np.abs(u[:, t]) * D + 4 * U * np.abs(hn)
        h = hn
        y[:, t], e_y[:, t] = h, err
    return {"y": y, "final": h, "states": np.stack(states, 1), "e_y": e_y, "e_final": err,
            "e_states": np.stack(e_states, 1)}


def gated_scan_bwd(x, gate_a, gate_x, decay, dy, init=None, reset=None, d_final=None, scale=8.0):
    """Gradients of sum(dy y) + sum(d_final final): dict dx, dgate_a, dgate_x,
    ddecay, d_init and e_*."""
    f = gated_scan(x, gate_a, gate_x, decay, init, reset, scale)
    x, gate_a, gate_x, decay, dy = map(_np, (x, gate_a, gate_x, decay, dy))
    init, reset, d_final = _np(init), _np(reset), _np(d_final)
    b, L, C = x.shape
    r, i, la, decays, em1, n = gates(gate_a, gate_x, decay, scale, reset)
    zero = np.zeros((b, C))
    hp = np.concatenate([(zero if init is None else init)[:, None], f["y"][:, :-1]], 1)
    e_hp = np.concatenate([zero[:, None], f["e_y"][:, :-1]], 1)
    carry = zero if d_final is None else d_final.copy()
    e_carry = np.zeros((b, C))
    o = {k: np.empty_like(x) for k in ("dx", "dgate_a", "dgate_x", "e_dx", "e_dgate_a", "e_dgate_x")}
    sums, e_sums, mags = np.zeros(C), np.zeros(C), np.zeros(C)
    for t in reversed(range(L)):
        g = dy[:, t] + carry
        e_g = e_carry + 2 * U * np.abs(g)
        on = np.ones((b, 1), bool) if reset is None else (reset[:, t] == 0)[:, None]
        a, nt, it = decays[:, t], n[:, t], i[:, t]
        # a = e^la with la off by D of itself: d(e^la) = a |la| D; and its own D
        e_a = a * (1.0 + np.abs(la[:, t])) * D + TINY
        ix = it * x[:, t]
        o["dx"][:, t] = g * nt * it
        o["e_dx"][:, t] = e_g * np.abs(nt * it) + D * np.abs(o["dx"][:, t])
        o["dgate_x"][:, t] = g * nt * ix * (1.0 - it)
        # 1 - i is formed from the rounded i: an absolute error
        o["e_dgate_x"][:, t] = (e_g * np.abs(nt * ix * (1.0 - it)) + D * np.abs(o["dgate_x"][:, t])
                                + D * np.abs(g * nt * ix))
        h_in = np.where(on, hp[:, t], 0.0)
        with np.errstate(divide="ignore", invalid="ignore"):
            per_a = np.where(on & (nt > 0), a / np.where(nt > 0, nt, 1.0) * np.abs(ix), 0.0)
            w = np.where(on & (nt > 0), a * a / np.where(nt > 0, nt, 1.0) * ix, 0.0)
        dla = np.where(on, g * (a * h_in - w), 0.0)
        e_dla = np.where(on, e_g * np.abs(a * h_in - w)
                         + np.abs(g) * (a * np.where(on, e_hp[:, t], 0.0) + D * (np.abs(a * h_in) + np.abs(w))
                                        + e_a * (np.abs(h_in) + 2.0 * per_a)), 0.0)
        k = la[:, t] * (1.0 - r[:, t])
        o["dgate_a"][:, t] = dla * k
        o["e_dgate_a"][:, t] = e_dla * np.abs(k) + D * np.abs(dla * la[:, t])
        sums += (dla * r[:, t]).sum(0)
        e_sums += (e_dla * r[:, t] + D * np.abs(dla * r[:, t])).sum(0)
        mags += np.abs(dla * r[:, t]).sum(0)
        c2 = np.where(on, a * np.where(on, g, 0.0), 0.0)
        e_carry = np.where(on, a * e_g + kept(la[:, t], a, em1[:, t], g) + 4 * U * np.abs(c2), 0.0)
        carry = c2
    ks = -scale * sigma(decay)
    o["ddecay"] = ks * sums
    o["e_ddecay"] = np.abs(ks) * (e_sums + U * b * L * mags) + D * np.abs(o["ddecay"])
    o["d_init"], o["e_d_init"] = carry, e_carry
    return o


def gated_state_update(state, x, gate_a, gate_x, decay, reset=None, scale=8.0):
    """One token: (new state, its error bound)."""
    one = [_np(v)[:, None] for v in (x, gate_a, gate_x)]
    f = gated_scan(*one, decay, state, None if reset is None else _np(reset)[:, None], scale)
    return f["final"], f["e_final"]


def _turn(v, ang, rot_dim, adjacent):
    """Rotates v's leading pairs by ang [..., rot_dim / 2]."""
    o = v.copy()
    half = rot_dim // 2
    for j in range(half):
        p, q = (2 * j, 2 * j + 1) if adjacent else (j, j + half)
        c, s = np.cos(ang[..., j]), np.sin(ang[..., j])
        o[..., p] = v[..., p] * c - v[..., q] * s
        o[..., q] = v[..., p] * s + v[..., q] * c
    return o


def _pair_size(v, rot_dim, adjacent):
    """|v_a| + |v_b| of each element's pair: what its rotation's error scales with."""
    v = np.abs(v)
    o = v.copy()
    half = rot_dim // 2
    for j in range(half):
        p, q = (2 * j, 2 * j + 1) if adjacent else (j, j + half)
        o[..., p] = o[..., q] = v[..., p] + v[..., q]
    return o


def _angles(positions, inv_freq, shape):
    b, L = shape
    pos = np.broadcast_to(np.arange(L), (b, L)) if positions is None else np.asarray(
        positions.cpu() if hasattr(positions, "cpu") else positions)
    f = np.zeros(0) if inv_freq is None else _np(inv_freq)
    # whole turns are taken off in extended precision
    ang = pos.astype(np.longdouble)[..., None] * f.astype(np.longdouble)
    tau = 2 * np.longdouble("3.14159265358979323846264338327950288")
    return np.asarray(ang - np.rint(ang / tau) * tau, dtype=np.float64)[:, :, None, :]


def norm_rope(v, weight, inv_freq, positions=None, eps=1e-5, adjacent=False):
    """One of q, k [b, L, H, D] -> (out, its error bound)."""
    v = _np(v)
    D_ = v.shape[-1]
    w = np.ones(D_) if weight is None else _np(weight)
    ang = _angles(positions, inv_freq, v.shape[:2])
    R = 2 * ang.shape[-1]
    u = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * w
    # the sum of squares adds up to D / 16 terms per lane, then a tree
    return _turn(u, ang, R, adjacent), (D + D_ * U / 8) * _pair_size(u, R, adjacent)


def norm_rope_bwd(v, weight, inv_freq, d_out, positions=None, eps=1e-5, adjacent=False):
    """-> dict dv, dweight and e_*."""
    v, d_out = _np(v), _np(d_out)
    b, L, H, D_ = v.shape
    w = np.ones(D_) if weight is None else _np(weight)
    ang = _angles(positions, inv_freq, v.shape[:2])
    R = 2 * ang.shape[-1]
    e = _turn(d_out, -ang, R, adjacent)
    s = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    m = (e * w * v).mean(-1, keepdims=True)
    dv = s * (e * w - v * s * s * m)
    de = (D + D_ * U / 8)
    size = _pair_size(d_out, R, adjacent) * np.abs(w)
    e_dv = 2 * de * s * (size + np.abs(v) * s * s * (size * np.abs(v)).mean(-1, keepdims=True))
    terms = e * v * s
    mag = (_pair_size(d_out, R, adjacent) * np.abs(v) * s).sum((0, 1, 2))
    return {"dv": dv, "e_dv": e_dv, "dweight": terms.sum((0, 1, 2)),
            "e_dweight": mag * (2 * de + U * b * L * H)}


def conv1d_bwd(x, weight, dy, bias=None, init=None, d_final=None, activation=True):
    """Gradients of the causal convolution -> dict dx, dweight, dbias, d_init, e_*."""
    x, w, dy, bias, init, d_final = map(_np, (x, weight, dy, bias, init, d_final))
    b, L, C = x.shape
    K = w.shape[1]
    carried = np.zeros((b, C, K - 1)) if init is None else init
    xin = np.concatenate([carried.transpose(0, 2, 1), x], 1)
    o = np.zeros((b, L, C)) if bias is None else np.broadcast_to(bias, (b, L, C)).copy()
    size = np.abs(o)
    for k in range(K):
        o = o + w[:, k] * xin[:, k:k + L]
        size = size + np.abs(w[:, k] * xin[:, k:k + L])
    d, e_d = dy.copy(), np.zeros_like(dy)
    if activation:
        sg = sigma(o)
        d = dy * sg * (1.0 + o * (1.0 - sg))
        # |silu''| <= 1/2 carries the sum's error; the factor's own terms are at most
        # 1 + |o|, each within 16 roundings
        e_d = np.abs(dy) * (0.5 * (K + 1) * U * size + D * (1.0 + np.abs(o)) * sg) + 2 * U * np.abs(d)
    dxin, e_in = np.zeros_like(xin), np.zeros_like(xin)
    dw, e_dw = np.zeros((C, K)), np.zeros((C, K))
    for k in range(K):
        dxin[:, k:k + L] += w[:, k] * d
        e_in[:, k:k + L] += np.abs(w[:, k]) * (e_d + (K + 2) * U * np.abs(d))
        t = d * xin[:, k:k + L]
        dw[:, k] = t.sum((0, 1))
        e_dw[:, k] = (e_d * np.abs(xin[:, k:k + L])).sum((0, 1)) + U * (b * L + 2) * np.abs(t).sum((0, 1))
    if d_final is not None:
        dxin[:, L:] += d_final.transpose(0, 2, 1)
        e_in += 2 * U * np.abs(dxin)
    return {"dx": dxin[:, K - 1:], "e_dx": e_in[:, K - 1:], "dweight": dw, "e_dweight": e_dw,
            "dbias": d.sum((0, 1)), "e_dbias": e_d.sum((0, 1)) + U * (b * L + 2) * np.abs(d).sum((0, 1)),
            "d_init": dxin[:, :K - 1].transpose(0, 2, 1), "e_d_init": e_in[:, :K - 1].transpose(0, 2, 1)}
