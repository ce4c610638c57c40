"""The C ABI and the binding of the gated recurrence, the head norm with the
rotation and the convolution's gradient refuse what they do not take, before
anything is launched (CPU only)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from mamba_ssd_scan_b200 import build
    build.build()
    import mamba_ssd_scan_b200 as m
    return m.load_library()


def _structs():
    import mamba_ssd_scan_b200 as m
    return {"ssd_conv1d_bwd_args": m.SsdConv1dBwdArgs, "ssd_gated_scan_args": m.SsdGatedScanArgs,
            "ssd_gated_scan_bwd_args": m.SsdGatedScanBwdArgs,
            "ssd_gated_state_update_args": m.SsdGatedStateUpdateArgs,
            "ssd_qk_norm_rope_args": m.SsdQkNormRopeArgs,
            "ssd_qk_norm_rope_bwd_args": m.SsdQkNormRopeBwdArgs}


def test_structs_mirror_the_header(tmp_path):
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"ssd.h\"\nint main(void){\n"
    for n, c in _structs().items():
        src += f'printf("{n} %zu",sizeof({n}));'
        src += "".join(f'printf(" %zu",offsetof({n},{f[0]}));' for f in c._fields_) + 'printf("\\n");\n'
    (tmp_path / "o.c").write_text(src + "return 0;}")
    exe = str(tmp_path / "o")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "o.c"), "-o", exe])
    lines = subprocess.check_output([exe]).decode().splitlines()
    assert len(lines) == len(_structs())
    for line in lines:
        n, *v = line.split()
        c = _structs()[n]
        assert [int(i) for i in v] == [ctypes.sizeof(c)] + [getattr(c, f[0]).offset for f in c._fields_], n
    import mamba_ssd_scan_b200 as m
    text = open(os.path.join(ROOT, "include", "ssd.h")).read()
    assert int(re.search(r"#define SSD_GATED_SCAN_INTERVAL (\d+)", text).group(1)) == m.SSD_GATED_SCAN_INTERVAL


GATED = dict(batch=2, seqlen=70, channels=16, dtype=1, scale=8.0)


@pytest.mark.parametrize("bad,status", [
    ({}, 1), (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(channels=-8), 1), (dict(dtype=2), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(channels=12), 2), (dict(dtype=0, channels=6), 2),
    (dict(batch=65536), 2), (dict(seqlen=1 << 31), 2), (dict(channels=1 << 31), 2),
])
def test_gated_scan_refusals(lib, bad, status):
    import mamba_ssd_scan_b200 as m
    kw = {**GATED, **bad}
    assert lib.ssd_gated_scan(ctypes.byref(m.SsdGatedScanArgs(**kw)), None) == status
    a = m.SsdGatedScanBwdArgs(**kw)
    assert lib.ssd_gated_scan_bwd(ctypes.byref(a), None) == status
    assert (lib.ssd_gated_scan_bwd_workspace_size(ctypes.byref(a)) > 0) == (bad == {})
    if "seqlen" not in bad:
        kw.pop("seqlen")
        assert lib.ssd_gated_state_update(ctypes.byref(m.SsdGatedStateUpdateArgs(**kw)), None) == status
    assert lib.ssd_gated_scan(None, None) == lib.ssd_gated_scan_bwd(None, None) == 1
    assert lib.ssd_gated_state_update(None, None) == 1
    assert lib.ssd_gated_scan_bwd_workspace_size(None) == 0


QK = dict(batch=2, seqlen=7, q_heads=4, k_heads=2, headdim=64, rot_dim=64, dtype=1, eps=1e-5)
QK_STRIDES = dict(q_stride=256, k_stride=128)


@pytest.mark.parametrize("bad,status", [
    ({}, 1), (dict(batch=0), 1), (dict(q_heads=0), 1), (dict(k_heads=-1), 1), (dict(headdim=0), 1),
    (dict(rot_dim=80), 1), (dict(rot_dim=-16), 1), (dict(dtype=5), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(headdim=60, rot_dim=0), 2), (dict(headdim=264), 2),
    (dict(rot_dim=24), 2), (dict(q_heads=65536), 2), (dict(batch=1 << 20, seqlen=1 << 11), 2),
    (dict(batch=1 << 40, seqlen=1 << 40), 2),
    (dict(q_stride=248), 1), (dict(k_stride=0), 1), (dict(q_stride=260), 2), (dict(q_stride=1 << 31), 2),
])
def test_qk_norm_rope_refusals(lib, bad, status):
    import mamba_ssd_scan_b200 as m
    kw = {**QK, **QK_STRIDES, **bad}
    f = dict(kw, q_out_stride=kw["q_stride"], k_out_stride=kw["k_stride"])
    assert lib.ssd_qk_norm_rope(ctypes.byref(m.SsdQkNormRopeArgs(**f)), None) == status
    for name in ("q_stride", "dq_out_stride", "dq_stride"):  # each of the backward's strides
        w = {**QK, "q_stride": 256, "dq_out_stride": 256, "dq_stride": 256, "k_stride": kw["k_stride"],
             "dk_out_stride": 128, "dk_stride": 128, **{k: v for k, v in bad.items() if k != "q_stride"}}
        w[name] = kw["q_stride"]
        a = m.SsdQkNormRopeBwdArgs(**w)
        assert lib.ssd_qk_norm_rope_bwd(ctypes.byref(a), None) == status, name
    strides = any("stride" in k for k in bad)
    assert (lib.ssd_qk_norm_rope_bwd_workspace_size(ctypes.byref(a)) > 0) == (bad == {} or strides)
    assert lib.ssd_qk_norm_rope(None, None) == lib.ssd_qk_norm_rope_bwd(None, None) == 1
    assert lib.ssd_qk_norm_rope_bwd_workspace_size(None) == 0


@pytest.mark.parametrize("bad,status", [
    ({}, 1), (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(width=0), 1), (dict(dtype=2), 1),
    (dict(width=9), 2), (dict(channels=12), 2), (dict(dtype=0, channels=6), 2), (dict(batch=65536), 2),
    (dict(seqlen=1 << 31), 2),
])
def test_conv1d_bwd_refusals(lib, bad, status):
    import mamba_ssd_scan_b200 as m
    a = m.SsdConv1dBwdArgs(**{**dict(batch=2, seqlen=70, channels=16, width=4, dtype=1), **bad})
    assert lib.ssd_causal_conv1d_bwd(ctypes.byref(a), None) == status
    assert (lib.ssd_causal_conv1d_bwd_workspace_size(ctypes.byref(a)) > 0) == (bad == {})
    assert lib.ssd_causal_conv1d_bwd(None, None) == 1
    assert lib.ssd_causal_conv1d_bwd_workspace_size(None) == 0


def test_host_memory_is_refused(lib):
    import mamba_ssd_scan_b200 as m
    buf = torch.zeros(1 << 16)
    p = buf.data_ptr()
    ws = dict(workspace=p, workspace_bytes=1 << 17)
    g = dict(GATED, x=p, gate_a=p, gate_x=p, decay=p)
    assert lib.ssd_gated_scan(ctypes.byref(m.SsdGatedScanArgs(**g, y=p)), None) == 1
    assert lib.ssd_gated_scan_bwd(ctypes.byref(m.SsdGatedScanBwdArgs(
        **g, states=p, dy=p, dx=p, dgate_a=p, dgate_x=p, ddecay=p, **ws)), None) == 1
    a = m.SsdQkNormRopeArgs(**QK, **QK_STRIDES, q_out_stride=256, k_out_stride=128, q=p, k=p, q_out=p,
                            k_out=p, inv_freq=p)
    assert lib.ssd_qk_norm_rope(ctypes.byref(a), None) == 1
    c = m.SsdConv1dBwdArgs(batch=1, seqlen=8, channels=8, width=2, dtype=1, x=p, weight=p, dy=p, dx=p,
                           dweight=p, **ws)
    assert lib.ssd_causal_conv1d_bwd(ctypes.byref(c), None) == 1


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_checks_shapes_and_types(lib):
    import mamba_ssd_scan_b200 as m
    x, d = _bf(2, 70, 16), torch.zeros(16)
    for kw, exc in ((dict(gate_a=_bf(2, 69, 16)), ValueError), (dict(gate_x=x.float()), TypeError),
                    (dict(decay=torch.zeros(15)), ValueError), (dict(decay=_bf(16)), TypeError),
                    (dict(init_state=torch.zeros(2, 15)), ValueError),
                    (dict(reset=torch.zeros(2, 71, dtype=torch.uint8)), ValueError),
                    (dict(reset=torch.zeros(2, 70)), TypeError),
                    (dict(states=torch.zeros(2, 1, 16)), ValueError),
                    (dict(gate_a=_bf(2, 16, 70).transpose(1, 2)), ValueError),
                    ({}, m.SsdError)):  # host memory: the library's own refusal
        with pytest.raises(exc):
            m.ssd_gated_scan(**{**dict(x=x, gate_a=x, gate_x=x, decay=d), **kw})
    st = torch.zeros(2, 2, 16)
    for kw, exc in ((dict(dy=_bf(2, 70, 8)), ValueError), (dict(states=torch.zeros(2, 3, 16)), ValueError),
                    (dict(out={"dx": _bf(2, 70, 8)}), ValueError),
                    (dict(workspace=torch.zeros(4)), ValueError), ({}, m.SsdError)):
        with pytest.raises(exc):
            m.ssd_gated_scan_bwd(**{**dict(x=x, gate_a=x, gate_x=x, decay=d, dy=x, states=st), **kw})
    s1, x1 = torch.zeros(2, 16), _bf(2, 16)
    for kw, exc in ((dict(state=_bf(2, 16)), TypeError), (dict(new_state=torch.zeros(1, 16)), ValueError),
                    (dict(reset=torch.zeros(3, dtype=torch.bool)), ValueError), ({}, m.SsdError)):
        with pytest.raises(exc):
            m.ssd_gated_state_update(**{**dict(state=s1, x=x1, gate_a=x1, gate_x=x1, decay=d), **kw})
    q, k, w, f = _bf(2, 7, 4, 64), _bf(2, 7, 2, 64), torch.ones(64), torch.ones(32)
    base = dict(q=q, k=k, q_weight=w, k_weight=w, inv_freq=f)
    for kw, exc in ((dict(k=_bf(2, 6, 2, 64)), ValueError), (dict(k=k.float()), TypeError),
                    (dict(q_weight=torch.ones(63)), ValueError), (dict(inv_freq=torch.ones(33)), m.SsdError),
                    (dict(positions=torch.zeros(2, 7)), TypeError),
                    (dict(positions=torch.zeros(7, dtype=torch.int64)), ValueError),
                    (dict(q=_bf(2, 4, 7, 64).transpose(1, 2)), ValueError),      # heads not dense
                    (dict(q=_bf(2, 9, 4, 64)[:, :7]), ValueError),               # uneven tokens
                    (dict(q=_bf(2, 1, 4, 64).expand(2, 7, 4, 64)), ValueError),  # broadcast
                    (dict(q_out=_bf(2, 7, 4, 32)), ValueError), ({}, m.SsdError)):
        with pytest.raises(exc):
            m.ssd_qk_norm_rope(**{**base, **kw})
        if "q_out" not in kw:
            with pytest.raises(exc):
                m.ssd_qk_norm_rope_bwd(**{**base, "dq_out": q, "dk_out": k, **kw})
    with pytest.raises(ValueError):
        m.ssd_qk_norm_rope_bwd(**base, dq_out=_bf(2, 7, 4, 32), dk_out=k)
    xw = torch.zeros(16, 4)
    for kw, exc in ((dict(weight=torch.zeros(15, 4)), ValueError), (dict(dy=_bf(2, 71, 16)), ValueError),
                    (dict(bias=torch.zeros(1)), ValueError), (dict(d_final=torch.zeros(2, 16, 4)), ValueError),
                    (dict(weight=torch.zeros(16, 9)), m.SsdError), ({}, m.SsdError)):
        with pytest.raises(exc):
            m.ssd_causal_conv1d_bwd(**{**dict(x=x, weight=xw, dy=x), **kw})


def test_streams_and_devices_that_do_not_match_are_refused(monkeypatch):
    """Nothing is launched unless the tensors, the stream and the current device
    are the same one."""
    import types
    import mamba_ssd_scan_b200 as m
    calls = []
    entry = types.SimpleNamespace(name="entry", pack=lambda *a: b"",
                                  fn=lambda args, handle: calls.append(handle) or 0)

    def stream(index):
        return types.SimpleNamespace(cuda_stream=1000 + index, device_index=index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for s, dev in ((None, 1), (stream(1), 1), (stream(0), 1), (stream(1), 0), (None, -1), (stream(0), -1)):
        with pytest.raises(m.SsdError):
            m._call(entry, s, dev)
    assert not calls
    m._call(entry, stream(0), 0)
    assert calls == [1000]
