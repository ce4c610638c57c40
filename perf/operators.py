"""What is timed and compared for the gated linear recurrence, the head norm with
the position rotation, and the gradient of the causal convolution: the cases,
their inputs, each operator in plain torch operations, and each operator's
definition in 64 bits.

With ``own`` false ``run`` computes the plain forms; with ``own`` true it makes
the calls of ``mamba_ssd_scan_b200`` that a user makes.

The operators, per element (sigma is the logistic function):

  scan     log a_t = -scale * softplus(decay_c) * sigma(gate_a_t), a_t = 0 where a
           sequence restarts;  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigma(gate_x_t) x_t;
           y_t = h_t.  The states entering every 64th token are kept for the gradient.
  scan_bwd the gradients of sum(dy * y) + sum(d_final * h_L) of the same.
  update   one token of the same against a carried state.
  rot      RMSNorm over each head of q and k times a weight, then the rotation of
           the pairs of the first 2 * len(inv_freq) elements by position * inv_freq.
  rot_bwd  its gradients.
  conv_bwd the gradients of the causal depthwise convolution (+ SiLU).
"""
import math

import torch

own = False

DEV = "cuda"
SCALE = 8.0
EPS = 1e-5
INTERVAL = 64  # tokens between the states the scan keeps for its gradient


# ---- the cases ---------------------------------------------------------------
def listed():
    return [
        # one long prompt through one layer, 24 heads of 64 channels wide
        {"name": "scan_bf16_b1_L65536_C1536", "op": "scan", "dtype": "bf16", "b": 1, "L": 65536,
         "C": 1536, "resets": 0, "init": False},
        # packed documents in fp32, ragged length, channels that fill no whole tile
        {"name": "scan_f32_b3_L1000_C260", "op": "scan", "dtype": "f32", "b": 3, "L": 1000,
         "C": 260, "resets": 7, "init": True},
        # a training step's layer: 32 heads of 64 channels, eight sequences
        {"name": "scan_bwd_bf16_b8_L4096_C2048", "op": "scan_bwd", "dtype": "bf16", "b": 8,
         "L": 4096, "C": 2048, "resets": 0, "init": False},
        # fine-tuning on packed short documents in fp32
        {"name": "scan_bwd_f32_b2_L777_C1536", "op": "scan_bwd", "dtype": "f32", "b": 2, "L": 777,
         "C": 1536, "resets": 5, "init": True},
        # one new token for a full decode batch, 80 heads of 64 channels
        {"name": "update_bf16_b256_C5120", "op": "update", "dtype": "bf16", "b": 256, "C": 5120,
         "resets": 0},
        # one new token for a single sequence: latency only
        {"name": "update_f32_b1_C1536", "op": "update", "dtype": "f32", "b": 1, "C": 1536,
         "resets": 0},
        # C and B of a long prompt (8 groups, state 128), read in place from the
        # convolution's output beside 80 heads of 64 channels of x
        {"name": "rot_bf16_b1_L65536_G8_N128", "op": "rot", "dtype": "bf16", "b": 1, "L": 65536,
         "hq": 8, "hk": 8, "D": 128, "R": 128, "lead": 5120, "adjacent": False, "far": 0},
        # one new token for a decode batch at scattered far positions, shared key heads
        {"name": "rot_bf16_b256_L1_H32_K8_D64", "op": "rot", "dtype": "bf16", "b": 256, "L": 1,
         "hq": 32, "hk": 8, "D": 64, "R": 64, "lead": 0, "adjacent": False, "far": 1000000},
        # the gradient of the same in training, shared key heads
        {"name": "rot_bwd_bf16_b4_L4096_H32_K8_D128", "op": "rot_bwd", "dtype": "bf16", "b": 4,
         "L": 4096, "hq": 32, "hk": 8, "D": 128, "R": 128, "lead": 0, "adjacent": False, "far": 0},
        # a ragged fp32 batch, only part of each head rotated, adjacent pairs
        {"name": "rot_bwd_f32_b3_L501_H4_K2_D80", "op": "rot_bwd", "dtype": "f32", "b": 3,
         "L": 501, "hq": 4, "hk": 2, "D": 80, "R": 32, "lead": 0, "adjacent": True, "far": 5000},
        # the convolution in front of the scan in training: x, B and C of 32 heads of
        # 64 channels with one group of state 128
        {"name": "conv_bwd_bf16_b8_L4096_C2304_K4", "op": "conv_bwd", "dtype": "bf16", "b": 8,
         "L": 4096, "C": 2304, "K": 4, "act": True, "init": False},
        # a ragged fp32 batch that continues earlier sequences, no activation
        {"name": "conv_bwd_f32_b2_L1001_C260_K3", "op": "conv_bwd", "dtype": "f32", "b": 2,
         "L": 1001, "C": 260, "K": 3, "act": False, "init": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges: any operator, both types, sizes spread over
    their logarithm, odd ones among them, at most 64 Mi elements."""
    op = rng.choice(["scan", "scan_bwd", "update", "rot", "rot_bwd", "conv_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = 8 if dtype == "bf16" else 4
    cap = (1 << 26) if dtype == "bf16" else (1 << 25)
    if op == "update":
        return {"op": op, "dtype": dtype, "b": _log_int(rng, 1, 512),
                "C": step * _log_int(rng, 2, 5120 // step), "resets": rng.choice([0, 0, 1])}
    if op in ("rot", "rot_bwd"):
        D = rng.choice([32, 64, 80, 96, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 5])
        b = _log_int(rng, 1, 256)
        L = _log_int(rng, 1, min(65536, max(1, cap // 2 // (b * D * (hq + hk)))))
        return {"op": op, "dtype": dtype, "b": b, "L": L, "hq": hq, "hk": hk, "D": D,
                "R": rng.choice([D, D, D // 2 // 16 * 16]), "lead": rng.choice([0, 0, 64 * hq]),
                "adjacent": rng.random() < 0.3, "far": rng.choice([0, 0, 5000, 1000000])}
    C = step * _log_int(rng, 2, 5120 // step)
    b = _log_int(rng, 1, 64)
    L = _log_int(rng, 1, min(65536, max(1, cap // 2 // (b * C))))
    case = {"op": op, "dtype": dtype, "b": b, "L": L, "C": C, "init": rng.random() < 0.5}
    if op == "conv_bwd":
        case.update(K=rng.choice([2, 3, 4, 4, 4, 5, 8]), act=rng.random() < 0.8)
    else:
        case.update(resets=rng.choice([0, 0, 3, 20]))
    return case


# ---- the inputs --------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1000003 * (seed + 1) + 17)
    dt = _dtype(case)

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    s = {"case": dict(case)}
    op, b = case["op"], case["b"]
    if op in ("scan", "scan_bwd", "update"):
        C = case["C"]
        lead = (b,) if op == "update" else (b, case["L"])
        s["x"], s["gate_a"], s["gate_x"] = normal(*lead, C), normal(*lead, C), normal(*lead, C)
        # softplus(decay) = -log(a0) / scale: the slowest decay a0 of a channel lies in
        # [0.9, 0.999], the usual initialisation of such gates
        s["decay"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * uniform(C)) / SCALE))
        s["reset"] = None
        if case["resets"]:
            s["reset"] = (uniform(*lead) < min(0.5, case["resets"] / lead[-1])).to(torch.uint8)
        if op == "update":
            s["state"], s["new_state"] = normal(b, C, dtype=torch.float32), torch.empty(b, C, device=DEV)
            s["y"] = torch.empty_like(s["x"])
            return s
        s["init_state"] = normal(b, C, dtype=torch.float32) if case["init"] else None
        if op == "scan_bwd":
            s["dy"] = normal(b, case["L"], C)
            s["d_final"] = normal(b, C, dtype=torch.float32) if case["init"] else None
            # what the training step's forward left behind
            s["states"] = _scan_plain(s)[2]
    elif op in ("rot", "rot_bwd"):
        L, hq, hk, D, R = case["L"], case["hq"], case["hk"], case["D"], case["R"]
        wide = case["lead"] + (hq + hk) * D

        def heads():
            # k and q lie behind `lead` other channels of one packed row (k first, as B
            # lies before C); read in place
            buf = normal(b, L, wide)
            k = buf[..., case["lead"]:case["lead"] + hk * D].unflatten(-1, (hk, D))
            q = buf[..., case["lead"] + hk * D:].unflatten(-1, (hq, D))
            return q, k

        s["q"], s["k"] = heads()
        s["q_weight"] = 1.0 + normal(D, std=0.1, dtype=torch.float32)
        s["k_weight"] = 1.0 + normal(D, std=0.1, dtype=torch.float32)
        s["inv_freq"] = None
        if R:
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(DEV)
        s["positions"] = None
        if case["far"]:
            first = torch.randint(0, case["far"], (b, 1), generator=g, device=DEV)
            s["positions"] = first + torch.arange(L, device=DEV)
        if op == "rot_bwd":
            s["dq_out"], s["dk_out"] = normal(b, L, hq, D), normal(b, L, hk, D)
    else:
        L, C, K = case["L"], case["C"], case["K"]
        s["x"], s["dy"] = normal(b, L, C), normal(b, L, C)
        s["weight"] = normal(C, K, std=K ** -0.5, dtype=torch.float32)
        s["bias"] = normal(C, std=0.1, dtype=torch.float32)
        s["init_state"] = normal(b, C, K - 1, dtype=torch.float32) if case["init"] else None
        s["d_final"] = normal(b, C, K - 1, dtype=torch.float32) if case["init"] else None
    return s


# ---- the plain forms ---------------------------------------------------------
def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension 1, by doubling."""
    d, L = 1, a.shape[1]
    while d < L:
        u = torch.cat([u[:, :d], u[:, d:] + a[:, d:] * u[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return u


def _gates(s):
    """sigma(gate_a), sigma(gate_x), log a, a, sqrt(1 - a^2) in fp32."""
    r, i = torch.sigmoid(s["gate_a"].float()), torch.sigmoid(s["gate_x"].float())
    decay = s["decay"].float()
    sp = torch.clamp(decay, min=0) + torch.log1p(torch.exp(-decay.abs()))
    la = -SCALE * sp * r
    a, n = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    if s["reset"] is not None:
        on = s["reset"].bool()[..., None]
        a, n = torch.where(on, torch.zeros_like(a), a), torch.where(on, torch.ones_like(n), n)
    return r, i, sp, a, n


def _scan_plain(s):
    r, i, sp, a, n = _gates(s)
    u = n * i * s["x"].float()
    h0 = s["init_state"] if s["init_state"] is not None else torch.zeros_like(u[:, 0])
    u = torch.cat([u[:, :1] + a[:, :1] * h0[:, None], u[:, 1:]], 1)
    h = _linear_scan(a, u)
    states = torch.cat([h0[:, None], h[:, INTERVAL - 1:-1:INTERVAL]], 1)
    return h.to(s["x"].dtype), h[:, -1].clone(), states.contiguous()


def _scan_bwd_plain(s):
    r, i, sp, a, n = _gates(s)
    x = s["x"].float()
    h0 = s["init_state"] if s["init_state"] is not None else torch.zeros_like(x[:, 0])
    u = n * i * x
    u = torch.cat([u[:, :1] + a[:, :1] * h0[:, None], u[:, 1:]], 1)
    h = _linear_scan(a, u)
    hp = torch.cat([h0[:, None], h[:, :-1]], 1)
    # dh_t = dy_t + a_{t+1} dh_{t+1}: the same scan over reversed tokens
    dy = s["dy"].float()
    if s["d_final"] is not None:
        dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["d_final"][:, None]], 1)
    an = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    dh = _linear_scan(an.flip(1), dy.flip(1)).flip(1)
    dx = dh * n * i
    dgx = dh * n * x * i * (1 - i)
    # d log a = dh (a h_{t-1} - a^2 / n * i x); nothing flows to a gate that a restart switched off
    dla = dh * (a * hp - a * a / torch.clamp(n, min=1e-18) * (i * x))
    dga = dla * (-SCALE * sp) * r * (1 - r)
    ddecay = (dla.double() * (-SCALE * torch.sigmoid(s["decay"])) * r).sum((0, 1)).float()
    dt = s["x"].dtype
    return [dx.to(dt), dga.to(dt), dgx.to(dt), ddecay, a[:, 0] * dh[:, 0]]


def _update_plain(s):
    r, i, sp, a, n = _gates(s)
    h = a * s["state"] + n * i * s["x"].float()
    return [h.to(s["x"].dtype), h]


def _cos_sin(s, b, L):
    """cos and sin of position * inv_freq, [b, L, 1, R / 2]; the angles in 64 bits."""
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(L, device=DEV).expand(b, L)
    ang = pos.double()[..., None, None] * s["inv_freq"].double()
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(v, cos, sin, adjacent):
    """Rotates the pairs of v's last dimension."""
    if adjacent:
        a, b = v[..., 0::2], v[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = v.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _rot_plain(s):
    out = []
    R = 0 if s["inv_freq"] is None else 2 * s["inv_freq"].numel()
    if R:
        cos, sin = _cos_sin(s, *s["q"].shape[:2])
    for v, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        f = v.float()
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
        if R:
            f = torch.cat([_rotate(f[..., :R], cos, sin, s["case"]["adjacent"]), f[..., R:]], -1)
        out.append(f.to(v.dtype))
    return out


def _rot_bwd_plain(s):
    out = []
    R = 0 if s["inv_freq"] is None else 2 * s["inv_freq"].numel()
    if R:
        cos, sin = _cos_sin(s, *s["q"].shape[:2])
    for v, w, d in ((s["q"], s["q_weight"], s["dq_out"]), (s["k"], s["k_weight"], s["dk_out"])):
        f, d = v.float(), d.float()
        if R:  # the transposed rotation: by the negative angle
            d = torch.cat([_rotate(d[..., :R], cos, -sin, s["case"]["adjacent"]), d[..., R:]], -1)
        inv = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        dn = d * w
        dv = inv * (dn - f * inv * inv * (dn * f).mean(-1, keepdim=True))
        dw = (d * f * inv).double().sum((0, 1, 2)).float()
        out += [dv.to(v.dtype), dw]
    return out


def _conv_bwd_plain(s):
    x, w = s["x"].float(), s["weight"]
    b, L, C = x.shape
    K = w.shape[1]
    init = s["init_state"]
    head = init.transpose(1, 2) if init is not None else x.new_zeros(b, K - 1, C)
    xin = torch.cat([head, x], 1)  # [b, L + K - 1, C]
    d = s["dy"].float()
    if s["case"]["act"]:
        o = s["bias"].expand(b, L, C)
        for j in range(K):
            o = o + w[:, j] * xin[:, j:j + L]
        sg = torch.sigmoid(o)
        d = d * sg * (1 + o * (1 - sg))
    dxin = torch.zeros_like(xin)
    dw = []
    for j in range(K):
        dxin[:, j:j + L] += w[:, j] * d
        dw.append((d * xin[:, j:j + L]).double().sum((0, 1)))
    if s["d_final"] is not None:
        dxin[:, L:] += s["d_final"].transpose(1, 2)
    return [dxin[:, K - 1:].to(s["x"].dtype), torch.stack(dw, 1).float(),
            d.double().sum((0, 1)).float(), dxin[:, :K - 1].transpose(1, 2).contiguous()]


# ---- one pass ----------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"scan": lambda z: list(_scan_plain(z)), "scan_bwd": _scan_bwd_plain,
                "update": _update_plain, "rot": _rot_plain, "rot_bwd": _rot_bwd_plain,
                "conv_bwd": _conv_bwd_plain}[op](s)
    import mamba_ssd_scan_b200 as ssd
    if op == "scan":
        return list(ssd.ssd_gated_scan(s["x"], s["gate_a"], s["gate_x"], s["decay"],
                                       s["init_state"], s["reset"], scale=SCALE,
                                       return_final_state=True, return_states=True))
    if op == "scan_bwd":
        o = ssd.ssd_gated_scan_bwd(s["x"], s["gate_a"], s["gate_x"], s["decay"], s["dy"],
                                   s["states"], s["reset"], s["d_final"], scale=SCALE)
        return [o["dx"], o["dgate_a"], o["dgate_x"], o["ddecay"], o["d_init"]]
    if op == "update":
        y = ssd.ssd_gated_state_update(s["state"], s["x"], s["gate_a"], s["gate_x"], s["decay"],
                                       s["reset"], scale=SCALE, y=s["y"], new_state=s["new_state"])
        return [y, s["new_state"]]
    if op == "rot":
        return list(ssd.ssd_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"],
                                         s["inv_freq"], s["positions"], eps=EPS,
                                         adjacent=case["adjacent"]))
    if op == "rot_bwd":
        o = ssd.ssd_qk_norm_rope_bwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"],
                                     s["dq_out"], s["dk_out"], s["positions"], eps=EPS,
                                     adjacent=case["adjacent"])
        return [o["dq"], o["dq_weight"], o["dk"], o["dk_weight"]]
    o = ssd.ssd_causal_conv1d_bwd(s["x"], s["weight"], s["dy"], s["bias"], s["init_state"],
                                  s["d_final"], activation=case["act"])
    return [o["dx"], o["dweight"], o["dbias"], o["d_init"]]


# ---- what a pass cannot do without ------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, b = case["op"], case["b"]
    if op in ("rot", "rot_bwd"):
        rows = b * case["L"]
        n = rows * (case["hq"] + case["hk"]) * case["D"]
        small = 8 * case["D"] + 2 * case["R"] + (8 * rows if case["far"] else 0)
        if op == "rot":
            return {"bytes": 2 * e * n + small, "flops": 7 * n}
        return {"bytes": 3 * e * n + small + 8 * case["D"], "flops": 16 * n}
    C = case["C"]
    if op == "update":
        return {"bytes": (4 * e + 8) * b * C + 4 * C + (b if case["resets"] else 0), "flops": 20 * b * C}
    L = case["L"]
    n = b * L * C
    if op == "conv_bwd":
        K = case["K"]
        small = 8 * C * (K + 1) + (12 if case["init"] else 4) * b * C * (K - 1)
        return {"bytes": 3 * e * n + small, "flops": ((6 if case["act"] else 4) * K + (8 if case["act"] else 1)) * n}
    kept = 4 * b * C * -(-L // INTERVAL)
    small = 4 * C + (b * L if case["resets"] else 0)
    if op == "scan":
        return {"bytes": 4 * e * n + kept + small + (8 if case["init"] else 4) * b * C, "flops": 20 * n}
    return {"bytes": 7 * e * n + kept + small + 4 * C + (8 if case["init"] else 4) * b * C, "flops": 45 * n}


# ---- the definitions in 64 bits ----------------------------------------------
def _exact_scan(a, u, h):
    """h_t = a_t h_{t-1} + u_t from the state h: token by token inside blocks of tokens,
    all blocks at once from zero, then the blocks' carries one after the other."""
    b, L, C = u.shape
    m = max(1, int(math.isqrt(L)))
    nb = -(-L // m)
    pad = nb * m - L
    if pad:
        a = torch.cat([a, a.new_ones(b, pad, C)], 1)
        u = torch.cat([u, u.new_zeros(b, pad, C)], 1)
    a, u = a.view(b, nb, m, C), u.view(b, nb, m, C)
    loc, dec = torch.empty_like(u), torch.empty_like(u)
    loc[:, :, 0], dec[:, :, 0] = u[:, :, 0], a[:, :, 0]
    for t in range(1, m):
        loc[:, :, t] = a[:, :, t] * loc[:, :, t - 1] + u[:, :, t]
        dec[:, :, t] = a[:, :, t] * dec[:, :, t - 1]
    for k in range(nb):
        loc[:, k] += dec[:, k] * h[:, None]
        h = loc[:, k, -1]
    return loc.view(b, nb * m, C)[:, :L]


def _exact_recurrence(s):
    """The decay, the input weight's parts and their logarithms in fp64."""
    ga, gx, x = s["gate_a"].double(), s["gate_x"].double(), s["x"].double()
    dec = s["decay"].double()
    c = SCALE * torch.where(dec > 30, dec, torch.log1p(torch.exp(torch.clamp(dec, max=30))))
    r, i = 1 / (1 + torch.exp(-ga)), 1 / (1 + torch.exp(-gx))
    keep = torch.ones_like(x[..., :1])
    if s["reset"] is not None:
        keep = 1 - s["reset"].double()[..., None]
    a = torch.exp(-c * r) * keep
    n2 = torch.where(keep > 0, -torch.expm1(-2 * c * r), torch.ones_like(a))
    return a, n2.sqrt(), r, i, x, c, keep


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "update":
        a, n, r, i, x, c, keep = _exact_recurrence(s)
        h = a * s["state"].double() + n * i * x
        return [h, h]
    if op in ("scan", "scan_bwd"):
        b, L, C = s["x"].shape
        a, n, r, i, x, c, keep = _exact_recurrence(s)
        h0 = s["init_state"].double() if case["init"] else x.new_zeros(b, C)
        h = _exact_scan(a, n * i * x, h0)
        if op == "scan":
            at = [t - 1 for t in range(INTERVAL, L, INTERVAL)]
            return [h, h[:, -1], torch.cat([h0[:, None], h[:, at]], 1)]
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        # the adjoint g_t of h_t runs backwards: g_t = dy_t + a_{t+1} g_{t+1}
        after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
        last = s["d_final"].double() if case["init"] else x.new_zeros(b, C)
        g = _exact_scan(after.flip(1), s["dy"].double().flip(1), last).flip(1)
        # h = a h' + n v with v = i x, n = sqrt(1 - a^2), dn/da = -a / n, da/dr = -c a
        v = i * x
        da = g * (before - a / n * v) * keep
        dr = da * (-c * a)
        sg = 1 / (1 + torch.exp(-s["decay"].double()))
        ddecay = (da * a * -SCALE * r).sum((0, 1)) * sg
        dv = g * n
        return [dv * i, dr * r * (1 - r), dv * x * i * (1 - i), ddecay, a[:, 0] * g[:, 0]]
    if op in ("rot", "rot_bwd"):
        b, L = s["q"].shape[:2]
        D, R = case["D"], case["R"]
        # the rotation as complex numbers, one per pair
        pos = s["positions"] if case["far"] else torch.arange(L, device=DEV).expand(b, L)
        if R:
            ang = pos.double()[:, :, None, None] * s["inv_freq"].double()
            z = torch.complex(torch.cos(ang), torch.sin(ang))

        def turn(t, z):
            if not R:
                return t
            if case["adjacent"]:
                p = torch.view_as_complex(t[..., :R].reshape(*t.shape[:-1], R // 2, 2).contiguous()) * z
                p = torch.view_as_real(p).reshape(*t.shape[:-1], R)
            else:
                p = torch.complex(t[..., :R // 2].contiguous(), t[..., R // 2:R].contiguous()) * z
                p = torch.cat([p.real, p.imag], -1)
            return torch.cat([p, t[..., R:]], -1)

        out = []
        for name in ("q", "k"):
            f, w = s[name].double(), s[name + "_weight"].double()
            nrm = torch.sqrt(f.pow(2).sum(-1, keepdim=True) / D + EPS)
            if op == "rot":
                out.append(turn(f / nrm * w, z if R else None))
                continue
            g = turn(s["d" + name + "_out"].double(), z.conj() if R else None)
            unit = f / nrm
            gw = g * w
            out.append((gw - unit * ((gw * unit).sum(-1, keepdim=True) / D)) / nrm)
            out.append((g * unit).sum((0, 1, 2)))
        return out
    # the convolution's gradients, output token by input tap
    K, act = case["K"], case["act"]
    b, L, C = s["x"].shape
    w, dy = s["weight"].double(), s["dy"].double()
    ext = x_ext = torch.zeros(b, L + K - 1, C, dtype=torch.float64, device=DEV)
    x_ext[:, K - 1:] = s["x"].double()
    if case["init"]:
        x_ext[:, :K - 1] = s["init_state"].double().permute(0, 2, 1)
    win = ext.unfold(1, K, 1)  # [b, L, C, K], a view
    if act:
        o = torch.einsum("blck,ck->blc", win, w) + s["bias"].double()
        e = torch.exp(-o)
        dy = dy * (1 + e + o * e) / (1 + e) ** 2
    dw = torch.stack([(win[..., k] * dy).sum((0, 1)) for k in range(K)], 1)
    pad = torch.zeros(b, L + 2 * (K - 1), C, dtype=torch.float64, device=DEV)
    pad[:, K - 1:K - 1 + L] = dy
    back = torch.zeros_like(ext)
    for k in range(K):  # input j feeds output j - k through tap k
        back += pad[:, K - 1 - k:K - 1 - k + L + K - 1] * w[:, k]
    if case["init"]:
        back[:, L:] += s["d_final"].double().permute(0, 2, 1)
    return [back[:, K - 1:], dw, dy.sum((0, 1)), back[:, :K - 1].permute(0, 2, 1)]
