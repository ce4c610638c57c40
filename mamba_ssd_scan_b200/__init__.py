"""Mamba-2 SSD selective scan on NVIDIA B200: Python binding of libssd_b200.so.

The functions here carry the names of the C ABI in include/ssd.h and only
marshal arguments: they read shapes and device pointers off torch tensors,
allocate outputs/workspace with torch when the caller does not pass them, and
call the library on the current torch CUDA stream.  Every step of the scan runs
in the library's CUDA kernels; there is no CPU fallback, and a missing library
raises immediately.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

__all__ = [
    "SsdError", "ssd_fwd", "ssd_fwd_workspace_size", "ssd_fwd_check_status", "ssd_fwd_no_alloc",
    "ssd_fwd_no_alloc_check_status", "ssd_fwd_no_alloc_scratch_bytes", "ssd_debug_set_withhold",
    "SSD_DEBUG_CONV_TILE", "SSD_DEBUG_FWD_CARRY", "SSD_DEBUG_SCAN_DECAYS", "SSD_DEBUG_GATED_MAP",
    "ssd_fwd_tensor_core_steps", "tensor_core_steps", "ssd_chunk_cumsum", "ssd_chunk_state",
    "ssd_state_passing", "ssd_chunk_scan", "ssd_state_passing_hilo", "ssd_chunk_scan_hilo",
    "ssd_state_update", "ssd_status_string",
    "ssd_version", "lib_path", "load_library", "SSD_FLAG_CUDA_CORES", "SSD_FLAG_WHOLE_GROUPS",
    "SSD_FLAG_SPLIT_STEPS", "SSD_FLAG_BF16_STATES", "SSD_FLAG_SINGLE_PASS", "SSD_TC_CHUNK_STATE",
    "SSD_TC_CHUNK_SCAN",
    "SSD_TC_FUSED",
    "ssd_causal_conv1d", "ssd_conv1d_update", "ssd_conv1d_check_status",
    "ssd_bwd", "ssd_bwd_workspace_size", "ssd_selective_scan", "ssd_selective_scan_workspace_size",
    "ssd_selective_state_update", "ssd_gated_rmsnorm",
    "ssd_causal_conv1d_bwd", "ssd_causal_conv1d_bwd_workspace_size",
    "ssd_gated_scan", "ssd_gated_scan_bwd", "ssd_gated_scan_bwd_workspace_size",
    "ssd_gated_scan_check_status",
    "ssd_gated_state_update", "SSD_GATED_SCAN_INTERVAL",
    "ssd_qk_norm_rope", "ssd_qk_norm_rope_bwd", "ssd_qk_norm_rope_bwd_workspace_size",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_FILE = os.path.join(_PKG, "libssd_b200.so")

SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_CUDA, SSD_ERR_TIMEOUT = range(5)
SSD_F32, SSD_BF16 = 0, 1
SSD_FLAG_CUDA_CORES = 1
SSD_FLAG_WHOLE_GROUPS = 2
SSD_FLAG_SPLIT_STEPS = 4
SSD_FLAG_BF16_STATES = 8
SSD_FLAG_SINGLE_PASS = 16
SSD_TC_CHUNK_STATE, SSD_TC_CHUNK_SCAN, SSD_TC_FUSED = 1, 2, 4
SSD_GATED_SCAN_INTERVAL = 64

_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t


class SsdFwdArgs(ctypes.Structure):
    """Mirror of ssd_fwd_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("nheads", _i64), ("headdim", _i64),
                ("dstate", _i64), ("ngroups", _i64), ("chunk", _i64), ("dtype", _i32),
                ("flags", _i32), ("x", _vp), ("dt", _vp), ("A", _vp), ("B", _vp), ("C", _vp),
                ("D", _vp), ("dt_bias", _vp), ("init_state", _vp), ("y", _vp),
                ("final_state", _vp), ("workspace", _vp), ("workspace_bytes", _sz),
                ("z", _vp)]


class SsdBwdArgs(ctypes.Structure):
    """Mirror of ssd_bwd_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("nheads", _i64), ("headdim", _i64),
                ("dstate", _i64), ("ngroups", _i64), ("chunk", _i64), ("dtype", _i32),
                ("flags", _i32), ("x", _vp), ("dt", _vp), ("A", _vp), ("B", _vp), ("C", _vp),
                ("D", _vp), ("dt_bias", _vp), ("init_state", _vp), ("dy", _vp),
                ("d_final", _vp), ("dx", _vp), ("ddt", _vp), ("dA", _vp), ("dB", _vp),
                ("dC", _vp), ("dD", _vp), ("ddt_bias", _vp), ("d_init", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class SsdSelectiveScanArgs(ctypes.Structure):
    """Mirror of ssd_selective_scan_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("dstate", _i64),
                ("chunk", _i64), ("dtype", _i32), ("flags", _i32), ("x", _vp), ("dt", _vp),
                ("A", _vp), ("B", _vp), ("C", _vp), ("D", _vp), ("dt_bias", _vp),
                ("init_state", _vp), ("y", _vp), ("final_state", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class SsdSelectiveStateUpdateArgs(ctypes.Structure):
    """Mirror of ssd_selective_state_update_args."""
    _fields_ = [("batch", _i64), ("channels", _i64), ("dstate", _i64), ("dtype", _i32),
                ("flags", _i32), ("state", _vp), ("x", _vp), ("dt", _vp), ("A", _vp),
                ("B", _vp), ("C", _vp), ("D", _vp), ("dt_bias", _vp), ("y", _vp)]


class SsdStateUpdateArgs(ctypes.Structure):
    """Mirror of ssd_state_update_args."""
    _fields_ = [("batch", _i64), ("nheads", _i64), ("headdim", _i64), ("dstate", _i64),
                ("ngroups", _i64), ("dtype", _i32), ("flags", _i32), ("state", _vp),
                ("x", _vp), ("dt", _vp), ("A", _vp), ("B", _vp), ("C", _vp), ("D", _vp),
                ("dt_bias", _vp), ("y", _vp), ("z", _vp)]


class SsdConv1dArgs(ctypes.Structure):
    """Mirror of ssd_conv1d_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("width", _i64),
                ("dtype", _i32), ("activation", _i32), ("x", _vp), ("weight", _vp),
                ("bias", _vp), ("init_state", _vp), ("y", _vp), ("final_state", _vp)]


class SsdConv1dUpdateArgs(ctypes.Structure):
    """Mirror of ssd_conv1d_update_args."""
    _fields_ = [("batch", _i64), ("channels", _i64), ("width", _i64), ("dtype", _i32),
                ("activation", _i32), ("state", _vp), ("x", _vp), ("weight", _vp),
                ("bias", _vp), ("y", _vp)]


class SsdGatedRmsnormArgs(ctypes.Structure):
    """Mirror of ssd_gated_rmsnorm_args."""
    _fields_ = [("rows", _i64), ("channels", _i64), ("group", _i64), ("dtype", _i32),
                ("eps", ctypes.c_float), ("y", _vp), ("z", _vp), ("weight", _vp), ("out", _vp)]


class SsdConv1dBwdArgs(ctypes.Structure):
    """Mirror of ssd_conv1d_bwd_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("width", _i64),
                ("dtype", _i32), ("activation", _i32), ("x", _vp), ("weight", _vp),
                ("bias", _vp), ("init_state", _vp), ("dy", _vp), ("d_final", _vp), ("dx", _vp),
                ("dweight", _vp), ("dbias", _vp), ("d_init", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class SsdGatedScanArgs(ctypes.Structure):
    """Mirror of ssd_gated_scan_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("dtype", _i32),
                ("scale", ctypes.c_float), ("x", _vp), ("gate_a", _vp), ("gate_x", _vp),
                ("decay", _vp), ("reset", _vp), ("init_state", _vp), ("y", _vp),
                ("final_state", _vp), ("states", _vp)]


class SsdGatedScanBwdArgs(ctypes.Structure):
    """Mirror of ssd_gated_scan_bwd_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("dtype", _i32),
                ("scale", ctypes.c_float), ("x", _vp), ("gate_a", _vp), ("gate_x", _vp),
                ("decay", _vp), ("reset", _vp), ("states", _vp), ("dy", _vp), ("d_final", _vp),
                ("dx", _vp), ("dgate_a", _vp), ("dgate_x", _vp), ("ddecay", _vp),
                ("d_init", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class SsdGatedStateUpdateArgs(ctypes.Structure):
    """Mirror of ssd_gated_state_update_args."""
    _fields_ = [("batch", _i64), ("channels", _i64), ("dtype", _i32), ("scale", ctypes.c_float),
                ("state", _vp), ("x", _vp), ("gate_a", _vp), ("gate_x", _vp), ("decay", _vp),
                ("reset", _vp), ("new_state", _vp), ("y", _vp)]


class SsdQkNormRopeArgs(ctypes.Structure):
    """Mirror of ssd_qk_norm_rope_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("q_heads", _i64), ("k_heads", _i64),
                ("headdim", _i64), ("rot_dim", _i64), ("q_stride", _i64), ("k_stride", _i64),
                ("q_out_stride", _i64), ("k_out_stride", _i64), ("dtype", _i32),
                ("adjacent", _i32), ("eps", ctypes.c_float), ("q", _vp), ("k", _vp),
                ("q_weight", _vp), ("k_weight", _vp), ("inv_freq", _vp), ("positions", _vp),
                ("q_out", _vp), ("k_out", _vp)]


class SsdQkNormRopeBwdArgs(ctypes.Structure):
    """Mirror of ssd_qk_norm_rope_bwd_args."""
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("q_heads", _i64), ("k_heads", _i64),
                ("headdim", _i64), ("rot_dim", _i64), ("q_stride", _i64), ("k_stride", _i64),
                ("dq_out_stride", _i64), ("dk_out_stride", _i64), ("dq_stride", _i64),
                ("dk_stride", _i64), ("dtype", _i32), ("adjacent", _i32),
                ("eps", ctypes.c_float), ("q", _vp), ("k", _vp), ("q_weight", _vp),
                ("k_weight", _vp), ("inv_freq", _vp), ("positions", _vp), ("dq_out", _vp),
                ("dk_out", _vp), ("dq", _vp), ("dk", _vp), ("dq_weight", _vp),
                ("dk_weight", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class SsdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {ssd_status_string(status)}"
        if status == SSD_ERR_CUDA:
            msg += f" ({load_library().ssd_last_cuda_error().decode()})"
        super().__init__(msg)


_lib = None


def lib_path() -> str:
    return _LIB_FILE


def load_library():
    """Load libssd_b200.so (built by mamba_ssd_scan_b200.build); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_FILE):
        raise RuntimeError(f"{_LIB_FILE} is missing: run `python -m mamba_ssd_scan_b200.build`")
    lib = ctypes.CDLL(_LIB_FILE)
    F = ctypes.POINTER(SsdFwdArgs)
    lib.ssd_fwd_workspace_size.restype = _sz
    lib.ssd_fwd_workspace_size.argtypes = [F]
    lib.ssd_fwd.restype = ctypes.c_int
    lib.ssd_fwd.argtypes = [F, _vp]
    lib.ssd_fwd_tensor_core_steps.restype = ctypes.c_int
    lib.ssd_fwd_tensor_core_steps.argtypes = [F]
    lib.ssd_fwd_no_alloc.restype = ctypes.c_int
    lib.ssd_fwd_no_alloc.argtypes = [F, _vp]
    lib.ssd_fwd_check_status.restype = ctypes.c_int
    lib.ssd_fwd_check_status.argtypes = [F, _vp]
    lib.ssd_fwd_no_alloc_check_status.restype = ctypes.c_int
    lib.ssd_fwd_no_alloc_check_status.argtypes = [F, _vp]
    lib.ssd_fwd_no_alloc_scratch_bytes.restype = _sz
    lib.ssd_fwd_no_alloc_scratch_bytes.argtypes = []
    lib.ssd_debug_set_withhold.restype = None
    lib.ssd_debug_set_withhold.argtypes = [ctypes.c_int, ctypes.c_int64]
    lib.ssd_chunk_cumsum.restype = ctypes.c_int
    lib.ssd_chunk_cumsum.argtypes = [F, _vp, _vp, _vp]
    lib.ssd_chunk_state.restype = ctypes.c_int
    lib.ssd_chunk_state.argtypes = [F, _vp, _vp, _vp, _vp]
    lib.ssd_state_passing.restype = ctypes.c_int
    lib.ssd_state_passing.argtypes = [F, _vp, _vp, _vp]
    lib.ssd_chunk_scan.restype = ctypes.c_int
    lib.ssd_chunk_scan.argtypes = [F, _vp, _vp, _vp, _vp]
    lib.ssd_state_passing_hilo.restype = ctypes.c_int
    lib.ssd_state_passing_hilo.argtypes = [F, _vp, _vp, _vp, _vp]
    lib.ssd_chunk_scan_hilo.restype = ctypes.c_int
    lib.ssd_chunk_scan_hilo.argtypes = [F, _vp, _vp, _vp, _vp]
    lib.ssd_state_update.restype = ctypes.c_int
    lib.ssd_state_update.argtypes = [ctypes.POINTER(SsdStateUpdateArgs), _vp]
    BW = ctypes.POINTER(SsdBwdArgs)
    lib.ssd_bwd_workspace_size.restype = _sz
    lib.ssd_bwd_workspace_size.argtypes = [BW]
    lib.ssd_bwd.restype = ctypes.c_int
    lib.ssd_bwd.argtypes = [BW, _vp]
    lib.ssd_bwd_check_status.restype = ctypes.c_int
    lib.ssd_bwd_check_status.argtypes = [BW, _vp]
    SA = ctypes.POINTER(SsdSelectiveScanArgs)
    lib.ssd_selective_scan_workspace_size.restype = _sz
    lib.ssd_selective_scan_workspace_size.argtypes = [SA]
    lib.ssd_selective_scan.restype = ctypes.c_int
    lib.ssd_selective_scan.argtypes = [SA, _vp]
    lib.ssd_selective_state_update.restype = ctypes.c_int
    lib.ssd_selective_state_update.argtypes = [ctypes.POINTER(SsdSelectiveStateUpdateArgs), _vp]
    lib.ssd_causal_conv1d.restype = ctypes.c_int
    lib.ssd_causal_conv1d.argtypes = [ctypes.POINTER(SsdConv1dArgs), _vp]
    lib.ssd_conv1d_update.restype = ctypes.c_int
    lib.ssd_conv1d_update.argtypes = [ctypes.POINTER(SsdConv1dUpdateArgs), _vp]
    lib.ssd_gated_rmsnorm.restype = ctypes.c_int
    lib.ssd_gated_rmsnorm.argtypes = [ctypes.POINTER(SsdGatedRmsnormArgs), _vp]
    lib.ssd_causal_conv1d_bwd.restype = ctypes.c_int
    lib.ssd_causal_conv1d_bwd.argtypes = [ctypes.POINTER(SsdConv1dBwdArgs), _vp]
    lib.ssd_causal_conv1d_bwd_workspace_size.restype = _sz
    lib.ssd_causal_conv1d_bwd_workspace_size.argtypes = [ctypes.POINTER(SsdConv1dBwdArgs)]
    lib.ssd_gated_scan.restype = ctypes.c_int
    lib.ssd_gated_scan.argtypes = [ctypes.POINTER(SsdGatedScanArgs), _vp]
    lib.ssd_gated_scan_bwd.restype = ctypes.c_int
    lib.ssd_gated_scan_bwd.argtypes = [ctypes.POINTER(SsdGatedScanBwdArgs), _vp]
    lib.ssd_gated_scan_bwd_workspace_size.restype = _sz
    lib.ssd_gated_scan_bwd_workspace_size.argtypes = [ctypes.POINTER(SsdGatedScanBwdArgs)]
    lib.ssd_gated_state_update.restype = ctypes.c_int
    lib.ssd_gated_state_update.argtypes = [ctypes.POINTER(SsdGatedStateUpdateArgs), _vp]
    lib.ssd_qk_norm_rope.restype = ctypes.c_int
    lib.ssd_qk_norm_rope.argtypes = [ctypes.POINTER(SsdQkNormRopeArgs), _vp]
    lib.ssd_qk_norm_rope_bwd.restype = ctypes.c_int
    lib.ssd_qk_norm_rope_bwd.argtypes = [ctypes.POINTER(SsdQkNormRopeBwdArgs), _vp]
    lib.ssd_qk_norm_rope_bwd_workspace_size.restype = _sz
    lib.ssd_qk_norm_rope_bwd_workspace_size.argtypes = [ctypes.POINTER(SsdQkNormRopeBwdArgs)]
    lib.ssd_gated_scan_check_status.restype = ctypes.c_int
    lib.ssd_gated_scan_check_status.argtypes = [_vp]
    lib.ssd_conv1d_check_status.restype = ctypes.c_int
    lib.ssd_conv1d_check_status.argtypes = [_vp]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_last_cuda_error.restype = ctypes.c_char_p
    lib.ssd_last_cuda_error.argtypes = []
    lib.ssd_version.restype = ctypes.c_char_p
    lib.ssd_version.argtypes = []
    _lib = lib
    return lib


def ssd_status_string(status: int) -> str:
    return load_library().ssd_status_string(int(status)).decode()


def ssd_version() -> str:
    return load_library().ssd_version().decode()


# ---------------------------------------------------------------------------
def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SSD_F32
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != SSD_OK:
        raise SsdError(status, where)


def _fwd_args(x, dt, A, B, C, D, dt_bias, chunk, init_state, y, final_state, flags, z=None):
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    a = SsdFwdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, a.chunk = b, L, H, P, N, G, chunk
    a.dtype = _dtype_code(x)
    a.flags = int(flags)
    for name, t in (("dt", dt), ("B", B), ("C", C), ("z", z)):
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"{name} must have x's dtype {x.dtype}")
    if z is not None and tuple(z.shape) != tuple(x.shape):
        raise ValueError("z must have x's shape")
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias), ("init_state", init_state)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
    a.x, a.dt, a.A, a.B, a.C = _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C)
    a.D, a.dt_bias, a.init_state = _ptr(D), _ptr(dt_bias), _ptr(init_state)
    a.y, a.final_state = _ptr(y), _ptr(final_state)
    a.z = _ptr(z)
    return a


def ssd_fwd_workspace_size(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                           dtype=torch.bfloat16, flags: int = 0) -> int:
    a = SsdFwdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, a.chunk = (
        batch, seqlen, nheads, headdim, dstate, ngroups, chunk)
    a.dtype = SSD_BF16 if dtype == torch.bfloat16 else SSD_F32
    a.flags = flags
    return int(load_library().ssd_fwd_workspace_size(ctypes.byref(a)))


def ssd_fwd_tensor_core_steps(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                              dtype=torch.bfloat16, flags: int = 0) -> int:
    """Bitmask of the ssd_fwd steps that run on the tensor cores for these sizes
    (1 = chunk_state, 2 = chunk_scan, 4 = the whole forward as one kernel, with
    SSD_FLAG_SINGLE_PASS)."""
    a = SsdFwdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, a.chunk = (
        batch, seqlen, nheads, headdim, dstate, ngroups, chunk)
    a.dtype = SSD_BF16 if dtype == torch.bfloat16 else SSD_F32
    a.flags = flags
    return int(load_library().ssd_fwd_tensor_core_steps(ctypes.byref(a)))


def tensor_core_steps(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                      dtype=torch.bfloat16, flags: int = 0) -> set:
    """Names of the ssd_fwd steps that run on the tensor cores for these sizes."""
    m = ssd_fwd_tensor_core_steps(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                                  dtype, flags)
    return {n for bit, n in ((1, "chunk_state"), (2, "chunk_scan"), (4, "fused")) if m & bit}


def ssd_fwd(x, dt, A, B, C, D=None, dt_bias=None, chunk: int = 256, init_state=None, *,
            return_final_state: bool = False, y=None, final_state=None, workspace=None,
            flags: int = 0, stream=None, z=None):
    """The SSD scan forward.  x [b,L,H,P], dt [b,L,H] (raw), B/C [b,L,G,N] in one
    dtype (float32 or bfloat16); A, D, dt_bias [H] and init_state [b,H,P,N]
    float32; z (optional output gate, x's shape and dtype): y *= silu(z).
    Returns y (and the final fp32 state when asked)."""
    lib = load_library()
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and return_final_state:
        final_state = torch.empty((x.shape[0], x.shape[2], x.shape[3], B.shape[3]),
                                  dtype=torch.float32, device=x.device)
    a = _fwd_args(x, dt, A, B, C, D, dt_bias, chunk, init_state, y, final_state, flags, z)
    need = int(lib.ssd_fwd_workspace_size(ctypes.byref(a)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib.ssd_fwd(ctypes.byref(a), _stream_ptr(stream)), "ssd_fwd")
    if final_state is not None:
        return y, final_state
    return y


def _bwd_args(x, dt, A, B, C, D, dt_bias, chunk, init_state, flags):
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    a = SsdBwdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, a.chunk = b, L, H, P, N, G, chunk
    a.dtype = _dtype_code(x)
    a.flags = int(flags)
    for name, t in (("dt", dt), ("B", B), ("C", C)):
        if t.dtype != x.dtype:
            raise TypeError(f"{name} must have x's dtype {x.dtype}")
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias), ("init_state", init_state)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
    a.x, a.dt, a.A, a.B, a.C = _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C)
    a.D, a.dt_bias, a.init_state = _ptr(D), _ptr(dt_bias), _ptr(init_state)
    return a


def ssd_bwd_workspace_size(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                           dtype=torch.bfloat16, flags: int = 0) -> int:
    a = SsdBwdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, a.chunk = (
        batch, seqlen, nheads, headdim, dstate, ngroups, chunk)
    a.dtype = SSD_BF16 if dtype == torch.bfloat16 else SSD_F32
    a.flags = flags
    return int(load_library().ssd_bwd_workspace_size(ctypes.byref(a)))


def ssd_bwd(x, dt, A, B, C, dy, D=None, dt_bias=None, chunk: int = 256, init_state=None,
            d_final=None, *, out=None, workspace=None, flags: int = 0, stream=None) -> dict:
    """The backward pass of ssd_fwd (no output gate): gradients of
    sum(dy * y) + sum(d_final * final_state) with respect to every input.
    dy has x's shape and dtype; d_final [b,H,P,N] float32 or None.  Returns a
    dict dx, ddt (of the raw dt), dB, dC (input dtype), dA, dD, ddt_bias [H]
    and d_init [b,H,P,N] (float32); ``out`` may hold preallocated tensors under
    the same keys."""
    lib = load_library()
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    if dy.dtype != x.dtype or tuple(dy.shape) != tuple(x.shape):
        raise TypeError("dy must have x's shape and dtype")
    if d_final is not None and d_final.dtype != torch.float32:
        raise TypeError("d_final must be float32")
    o = dict(out or {})
    o.setdefault("dx", torch.empty_like(x))
    o.setdefault("ddt", torch.empty_like(dt))
    o.setdefault("dB", torch.empty_like(B))
    o.setdefault("dC", torch.empty_like(C))
    o.setdefault("dA", torch.empty(H, dtype=torch.float32, device=x.device))
    o.setdefault("dD", torch.empty(H, dtype=torch.float32, device=x.device))
    o.setdefault("ddt_bias", torch.empty(H, dtype=torch.float32, device=x.device))
    o.setdefault("d_init", torch.empty((b, H, P, N), dtype=torch.float32, device=x.device))
    a = _bwd_args(x, dt, A, B, C, D, dt_bias, chunk, init_state, flags)
    a.dy, a.d_final = _ptr(dy), _ptr(d_final)
    a.dx, a.ddt, a.dA, a.dB, a.dC = (_ptr(o["dx"]), _ptr(o["ddt"]), _ptr(o["dA"]), _ptr(o["dB"]),
                                     _ptr(o["dC"]))
    a.dD, a.ddt_bias, a.d_init = _ptr(o["dD"]), _ptr(o["ddt_bias"]), _ptr(o["d_init"])
    need = int(lib.ssd_bwd_workspace_size(ctypes.byref(a)))
    if need == 0:
        raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_bwd (sizes)")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib.ssd_bwd(ctypes.byref(a), _stream_ptr(stream)), "ssd_bwd")
    return o


SSD_DEBUG_CONV_TILE = 0
SSD_DEBUG_FWD_CARRY = 1
SSD_DEBUG_SCAN_DECAYS = 2
SSD_DEBUG_GATED_MAP = 3


def ssd_debug_set_withhold(what: int, index: int) -> None:
    """Test hook (include/ssd.h): make one producer withhold one hand-off so
    the consumers' bounded waits run out; index < 0 turns it off."""
    load_library().ssd_debug_set_withhold(int(what), int(index))


def ssd_fwd_no_alloc_scratch_bytes() -> int:
    """The size of the library's built-in scratch buffer (bytes)."""
    return int(load_library().ssd_fwd_no_alloc_scratch_bytes())


def ssd_fwd_no_alloc(x, dt, A, B, C, D=None, dt_bias=None, chunk: int = 256, init_state=None,
                     *, y, final_state=None, flags: int = 0, stream=None, z=None):
    """ssd_fwd without a workspace, for callers that cannot allocate: the
    scratch comes from a fixed buffer inside the library (see ssd_fwd_no_alloc
    in include/ssd.h).  ``y`` (and ``final_state``, if wanted) are caller-owned
    outputs; calls that can overlap on the GPU race and must be serialised.
    Sizes beyond the buffer are rejected by the library (SsdError,
    SSD_ERR_UNSUPPORTED) before anything is launched."""
    lib = load_library()
    a = _fwd_args(x, dt, A, B, C, D, dt_bias, chunk, init_state, y, final_state, flags, z)
    _check(lib.ssd_fwd_no_alloc(ctypes.byref(a), _stream_ptr(stream)), "ssd_fwd_no_alloc")
    return y


def ssd_fwd_no_alloc_check_status(x, B, chunk: int, flags: int = 0, stream=None) -> int:
    """Synchronise and return the device status of the last ssd_fwd_no_alloc
    call on the current device with these sizes (SSD_OK = 0,
    SSD_ERR_TIMEOUT = 4)."""
    b, L, H, P = x.shape
    a = SsdFwdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, a.chunk = (
        b, L, H, P, B.shape[3], B.shape[2], chunk)
    a.dtype = _dtype_code(x)
    a.flags = flags
    return int(load_library().ssd_fwd_no_alloc_check_status(ctypes.byref(a),
                                                            _stream_ptr(stream)))


def ssd_fwd_check_status(x, B, chunk: int, workspace, flags: int = 0, stream=None) -> int:
    """Synchronise and return the device status of the last ssd_fwd call that
    used ``workspace`` (SSD_OK = 0, SSD_ERR_TIMEOUT = 4)."""
    b, L, H, P = x.shape
    a = SsdFwdArgs()
    a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, a.chunk = (
        b, L, H, P, B.shape[3], B.shape[2], chunk)
    a.dtype = _dtype_code(x)
    a.flags = flags
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return int(load_library().ssd_fwd_check_status(ctypes.byref(a), _stream_ptr(stream)))


def _intermediate_shapes(x, B, chunk):
    b, L, H, P = x.shape
    N = B.shape[3]
    nc = (L + chunk - 1) // chunk
    return (b, H, nc, chunk), (b, nc, H, P, N)


def _states_dtype(x, flags):
    """The chunk states are fp32, except bf16 inputs in the bf16-states mode."""
    if x.dtype == torch.bfloat16 and flags & SSD_FLAG_BF16_STATES:
        return torch.bfloat16
    return torch.float32


def ssd_chunk_cumsum(x, dt, A, B, C, dt_bias=None, chunk: int = 256, *, dt_out=None,
                     cumA_out=None, stream=None):
    """Step 1: returns (dt, cumA), each [b, H, nc, chunk] float32."""
    lib = load_library()
    vshape, _ = _intermediate_shapes(x, B, chunk)
    dt_out = dt_out if dt_out is not None else torch.empty(vshape, dtype=torch.float32,
                                                           device=x.device)
    cumA_out = cumA_out if cumA_out is not None else torch.empty_like(dt_out)
    a = _fwd_args(x, dt, A, B, C, None, dt_bias, chunk, None, None, None, 0)
    _check(lib.ssd_chunk_cumsum(ctypes.byref(a), _ptr(dt_out), _ptr(cumA_out),
                                _stream_ptr(stream)), "ssd_chunk_cumsum")
    return dt_out, cumA_out


def ssd_chunk_state(x, dt, A, B, C, dt_sp, cumA, chunk: int = 256, *, states=None,
                    stream=None, flags: int = 0):
    """Step 2: returns the chunk-local states [b, nc, H, P, N], fp32 (bf16 for
    bf16 inputs with SSD_FLAG_BF16_STATES).  ``dt_sp``/``cumA`` are step 1's
    outputs."""
    lib = load_library()
    _, sshape = _intermediate_shapes(x, B, chunk)
    states = states if states is not None else torch.empty(
        sshape, dtype=_states_dtype(x, flags), device=x.device)
    a = _fwd_args(x, dt, A, B, C, None, None, chunk, None, None, None, flags)
    _check(lib.ssd_chunk_state(ctypes.byref(a), _ptr(dt_sp), _ptr(cumA), _ptr(states),
                               _stream_ptr(stream)), "ssd_chunk_state")
    return states


def ssd_state_passing(x, dt, A, B, C, cumA, states, chunk: int = 256, init_state=None,
                      final_state=None, stream=None, flags: int = 0):
    """Step 3, in place: ``states`` goes from chunk-local states to the states
    entering each chunk.  Writes ``final_state`` if given.  Returns states."""
    lib = load_library()
    a = _fwd_args(x, dt, A, B, C, None, None, chunk, init_state, None, final_state, flags)
    _check(lib.ssd_state_passing(ctypes.byref(a), _ptr(cumA), _ptr(states),
                                 _stream_ptr(stream)), "ssd_state_passing")
    return states


def ssd_chunk_scan(x, dt, A, B, C, dt_sp, cumA, states, D=None, chunk: int = 256, *, y=None,
                   stream=None, z=None, flags: int = 0):
    """Step 4: y from the chunk's tokens and the states entering each chunk
    (times silu(z) when the gate z is given)."""
    lib = load_library()
    y = y if y is not None else torch.empty_like(x)
    a = _fwd_args(x, dt, A, B, C, D, None, chunk, None, y, None, flags, z)
    _check(lib.ssd_chunk_scan(ctypes.byref(a), _ptr(dt_sp), _ptr(cumA), _ptr(states),
                              _stream_ptr(stream)), "ssd_chunk_scan")
    return y


def ssd_state_passing_hilo(x, dt, A, B, C, cumA, states, chunk: int = 256, init_state=None,
                           final_state=None, *, states_hl=None, stream=None, flags: int = 0):
    """Step 3 as ssd_fwd runs it for bf16 on the tensor cores: the fp32 local
    ``states`` (not modified) -> the states entering each chunk as hi / lo bf16
    halves, returned as ``states_hl`` [2, b, nc, H, P, N] (hi, then lo).
    Writes ``final_state`` if given."""
    lib = load_library()
    _, sshape = _intermediate_shapes(x, B, chunk)
    states_hl = states_hl if states_hl is not None else torch.empty(
        (2,) + sshape, dtype=torch.bfloat16, device=x.device)
    a = _fwd_args(x, dt, A, B, C, None, None, chunk, init_state, None, final_state, flags)
    _check(lib.ssd_state_passing_hilo(ctypes.byref(a), _ptr(cumA), _ptr(states), _ptr(states_hl),
                                      _stream_ptr(stream)), "ssd_state_passing_hilo")
    return states_hl


def ssd_chunk_scan_hilo(x, dt, A, B, C, dt_sp, cumA, states_hl, D=None, chunk: int = 256, *,
                        y=None, stream=None, z=None, flags: int = 0):
    """Step 4 on the tensor cores from the hi / lo entering states of
    ssd_state_passing_hilo (times silu(z) when the gate z is given)."""
    lib = load_library()
    y = y if y is not None else torch.empty_like(x)
    a = _fwd_args(x, dt, A, B, C, D, None, chunk, None, y, None, flags, z)
    _check(lib.ssd_chunk_scan_hilo(ctypes.byref(a), _ptr(dt_sp), _ptr(cumA), _ptr(states_hl),
                                   _stream_ptr(stream)), "ssd_chunk_scan_hilo")
    return y


def ssd_state_update(state, x, dt, A, B, C, D=None, dt_bias=None, *, y=None, stream=None,
                     z=None):
    """One decode step, in place on ``state`` [b,H,P,N] float32.  x [b,H,P],
    dt [b,H], B/C [b,G,N] in one dtype; z (optional output gate, x's shape and
    dtype).  Returns y [b,H,P] in x's dtype."""
    lib = load_library()
    b, H, P, N = state.shape
    G = B.shape[1]
    if state.dtype != torch.float32:
        raise TypeError("state must be float32")
    y = y if y is not None else torch.empty_like(x)
    a = SsdStateUpdateArgs()
    a.batch, a.nheads, a.headdim, a.dstate, a.ngroups = b, H, P, N, G
    a.dtype = _dtype_code(x)
    a.flags = 0
    a.state, a.x, a.dt, a.A, a.B, a.C = (_ptr(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
                                         _ptr(C))
    if z is not None and (z.dtype != x.dtype or tuple(z.shape) != tuple(x.shape)):
        raise TypeError("z must have x's shape and dtype")
    a.D, a.dt_bias, a.y, a.z = _ptr(D), _ptr(dt_bias), _ptr(y), _ptr(z)
    _check(lib.ssd_state_update(ctypes.byref(a), _stream_ptr(stream)), "ssd_state_update")
    return y


def ssd_causal_conv1d(x, weight, bias=None, init_state=None, *, activation: bool = True,
                      y=None, final_state=None, return_final_state: bool = False, stream=None):
    """Causal depthwise conv1d (+ SiLU) in front of the scan.  x [b,L,C] float32
    or bfloat16; weight [C,K] float32; bias [C] float32 or None; init_state
    [b,C,K-1] float32 or None.  Returns y (and the final [b,C,K-1] state when
    asked)."""
    lib = load_library()
    b, L, Cn = x.shape
    K = weight.shape[1]
    for name, t in (("weight", weight), ("bias", bias), ("init_state", init_state),
                    ("final_state", final_state)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
    y = y if y is not None else torch.empty_like(x)
    if final_state is None and return_final_state and K > 1:
        final_state = torch.empty((b, Cn, K - 1), dtype=torch.float32, device=x.device)
    a = SsdConv1dArgs()
    a.batch, a.seqlen, a.channels, a.width = b, L, Cn, K
    a.dtype = _dtype_code(x)
    a.activation = 1 if activation else 0
    a.x, a.weight, a.bias, a.init_state = _ptr(x), _ptr(weight), _ptr(bias), _ptr(init_state)
    a.y, a.final_state = _ptr(y), _ptr(final_state)
    _check(lib.ssd_causal_conv1d(ctypes.byref(a), _stream_ptr(stream)), "ssd_causal_conv1d")
    if return_final_state:
        return y, final_state
    return y


def _sel_args(x, dt, A, B, C, D, dt_bias, chunk, init_state, y, final_state):
    b, L, Dc = x.shape
    N = A.shape[1]
    for name, t in (("dt", dt), ("B", B), ("C", C)):
        if t.dtype != x.dtype:
            raise TypeError(f"{name} must have x's dtype {x.dtype}")
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias), ("init_state", init_state),
                    ("final_state", final_state)):
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
    a = SsdSelectiveScanArgs()
    a.batch, a.seqlen, a.channels, a.dstate, a.chunk = b, L, Dc, N, chunk
    a.dtype = _dtype_code(x)
    a.flags = 0
    a.x, a.dt, a.A, a.B, a.C = _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C)
    a.D, a.dt_bias, a.init_state = _ptr(D), _ptr(dt_bias), _ptr(init_state)
    a.y, a.final_state = _ptr(y), _ptr(final_state)
    return a


def ssd_selective_scan(x, dt, A, B, C, D=None, dt_bias=None, chunk: int = 64, init_state=None,
                       *, y=None, final_state=None, return_final_state: bool = False,
                       workspace=None, stream=None):
    """The diagonal-A (Mamba-1 form) selective scan.  x, dt [b,L,Dc] and B, C
    [b,L,N] in one dtype; A [Dc,N], D, dt_bias [Dc], init_state [b,Dc,N] fp32.
    Returns y (and the final fp32 state when asked)."""
    lib = load_library()
    b, L, Dc = x.shape
    N = A.shape[1]
    y = y if y is not None else torch.empty_like(x)
    if final_state is None and return_final_state:
        final_state = torch.empty((b, Dc, N), dtype=torch.float32, device=x.device)
    a = _sel_args(x, dt, A, B, C, D, dt_bias, chunk, init_state, y, final_state)
    need = int(lib.ssd_selective_scan_workspace_size(ctypes.byref(a)))
    if need == 0:
        raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_selective_scan (sizes)")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib.ssd_selective_scan(ctypes.byref(a), _stream_ptr(stream)), "ssd_selective_scan")
    if final_state is not None:
        return y, final_state
    return y


def ssd_selective_scan_workspace_size(batch, seqlen, channels, dstate, chunk,
                                      dtype=torch.bfloat16) -> int:
    a = SsdSelectiveScanArgs()
    a.batch, a.seqlen, a.channels, a.dstate, a.chunk = batch, seqlen, channels, dstate, chunk
    a.dtype = SSD_BF16 if dtype == torch.bfloat16 else SSD_F32
    return int(load_library().ssd_selective_scan_workspace_size(ctypes.byref(a)))


def ssd_selective_state_update(state, x, dt, A, B, C, D=None, dt_bias=None, *, y=None,
                               stream=None):
    """One decode step of the diagonal-A scan, in place on state [b,Dc,N] fp32;
    x, dt [b,Dc] and B, C [b,N] in one dtype.  Returns y [b,Dc]."""
    lib = load_library()
    b, Dc = x.shape
    N = A.shape[1]
    if state.dtype != torch.float32:
        raise TypeError("state must be float32")
    y = y if y is not None else torch.empty_like(x)
    a = SsdSelectiveStateUpdateArgs()
    a.batch, a.channels, a.dstate = b, Dc, N
    a.dtype = _dtype_code(x)
    a.flags = 0
    a.state, a.x, a.dt, a.A, a.B, a.C = (_ptr(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
                                         _ptr(C))
    a.D, a.dt_bias, a.y = _ptr(D), _ptr(dt_bias), _ptr(y)
    _check(lib.ssd_selective_state_update(ctypes.byref(a), _stream_ptr(stream)),
           "ssd_selective_state_update")
    return y


def ssd_conv1d_check_status(stream=None) -> int:
    """Synchronises the stream; SSD_ERR_TIMEOUT if a forward convolution on
    this device gave up on an internal wait since the last check, else 0."""
    return int(load_library().ssd_conv1d_check_status(_stream_ptr(stream)))


def ssd_conv1d_update(state, x, weight, bias=None, *, activation: bool = True, y=None,
                      stream=None):
    """One decode step of the convolution, in place on ``state`` [b,C,K-1]
    float32.  x [b,C].  Returns y [b,C] in x's dtype."""
    lib = load_library()
    b, Cn = x.shape
    K = weight.shape[1]
    if state is not None and state.dtype != torch.float32:
        raise TypeError("state must be float32")
    y = y if y is not None else torch.empty_like(x)
    a = SsdConv1dUpdateArgs()
    a.batch, a.channels, a.width = b, Cn, K
    a.dtype = _dtype_code(x)
    a.activation = 1 if activation else 0
    a.state, a.x, a.weight, a.bias, a.y = _ptr(state), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y)
    _check(lib.ssd_conv1d_update(ctypes.byref(a), _stream_ptr(stream)), "ssd_conv1d_update")
    return y


def ssd_gated_rmsnorm(y, z, weight, *, group: int | None = None, eps: float = 1e-5, out=None,
                      stream=None):
    """RMSNorm of g = y * silu(z) (g = y when z is None) over each group of
    ``group`` consecutive channels of the last axis (default: the whole last
    axis), times weight [channels] float32.  y, z: [..., channels] in one
    dtype.  ``out`` may be ``y`` (in place).  Returns out."""
    lib = load_library()
    channels = y.shape[-1]
    rows = y.numel() // channels
    if z is not None and (z.dtype != y.dtype or z.shape != y.shape):
        raise TypeError("z must match y in dtype and shape")
    if weight.dtype != torch.float32 or weight.numel() != channels:
        raise TypeError("weight must be float32 with one entry per channel")
    out = out if out is not None else torch.empty_like(y)
    a = SsdGatedRmsnormArgs()
    a.rows, a.channels, a.group = rows, channels, int(group if group is not None else channels)
    a.dtype = _dtype_code(y)
    a.eps = float(eps)
    a.y, a.z, a.weight, a.out = _ptr(y), _ptr(z), _ptr(weight), _ptr(out)
    _check(lib.ssd_gated_rmsnorm(ctypes.byref(a), _stream_ptr(stream)), "ssd_gated_rmsnorm")
    return out


# ---------------------------------------------------------------------------
# The gated linear recurrence, the head norm with the position rotation and the
# convolution's gradient.  Single-token steps and small batches are bound by the
# host, so these calls check each tensor once, pack their arguments with struct
# and read the stream's handle directly.
_CODES = {_i64: "q", _i32: "i", ctypes.c_float: "f", _vp: "P", _sz: "N"}


class _Entry:
    """A library function that takes one argument struct and a stream."""

    def __init__(self, lib, name, cls):
        self.name = name
        self.pack = struct.Struct("@" + "".join(_CODES[t] for _, t in cls._fields_) + "0q").pack
        self.fn = lib[name]  # a handle of its own, with its own prototype
        self.fn.restype = ctypes.c_int
        self.fn.argtypes = [ctypes.c_char_p, _vp]


def _entry(name, cls) -> _Entry:
    lib = load_library()
    try:
        return lib.entries[name]
    except (AttributeError, KeyError):
        if not hasattr(lib, "entries"):
            lib.entries = {}
        return lib.entries.setdefault(name, _Entry(lib, name, cls))


def _call(entry, stream, dev, *args):
    """Calls the entry with the struct's fields in order; dev is the tensors' device."""
    if dev < 0:
        raise SsdError(SSD_ERR_INVALID_ARG, entry.name + " (host memory)")
    if dev != torch.cuda.current_device():
        raise SsdError(SSD_ERR_INVALID_ARG, entry.name + " (tensors on another device than the current one)")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device_index == dev:
        handle = stream.cuda_stream
    else:
        raise SsdError(SSD_ERR_INVALID_ARG, entry.name + " (stream of another device than the tensors)")
    status = entry.fn(entry.pack(*args), handle)
    if status != SSD_OK:
        raise SsdError(status, entry.name)


def _addr(t, name, shape, dtype, dev) -> int:
    """The address of t, which must have this shape and dtype and lie, dense, on
    device number dev (-1 = host)."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    raise ValueError(f"{name} must be contiguous")


def _reset_addr(reset, shape, dev) -> int:
    if reset is None:
        return 0
    return _addr(reset, "reset", shape, torch.bool if reset.dtype is torch.bool else torch.uint8, dev)


@functools.lru_cache(maxsize=1024)
def _dense(shape):
    strides, n = [], 1
    for d in reversed(shape):
        strides.append(n)
        n *= d if d > 0 else 1
    return tuple(strides[::-1])


def _empty(shape, dtype, like, stream):
    """A dense tensor on like's device, from the pool of the stream that will write
    it, so that the allocator orders its reuse by that stream.  (empty_like takes
    half the time of empty, empty_strided two thirds.)"""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty(shape, dtype, like, None)
    if like.dtype is dtype and like.shape == shape and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty_strided(shape, _dense(shape), dtype=dtype, device=like.device)


def _output(given, name, shape, dtype, like, dev, stream):
    """An output tensor and its address: the caller's, checked, or a new one."""
    if given is None:
        t = _empty(shape, dtype, like, stream)
        return t, t.data_ptr()
    return given, _addr(given, name, shape, dtype, dev)


def _workspace(workspace, need, like, dev, stream):
    """(address, bytes) of the caller's workspace, or of a new one, and the tensor
    that keeps it."""
    if workspace is None:
        workspace = _empty((need,), torch.uint8, like, stream)
        return workspace.data_ptr(), need, workspace
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of the other tensors")
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace has {have} bytes, {need} are needed")
    return workspace.data_ptr(), have, workspace


_F32 = torch.float32


@functools.lru_cache(maxsize=1024)
def ssd_causal_conv1d_bwd_workspace_size(batch, seqlen, channels, width, dtype=torch.bfloat16) -> int:
    a = SsdConv1dBwdArgs(batch=batch, seqlen=seqlen, channels=channels, width=width,
                         dtype=SSD_BF16 if dtype == torch.bfloat16 else SSD_F32)
    return int(load_library().ssd_causal_conv1d_bwd_workspace_size(ctypes.byref(a)))


def ssd_causal_conv1d_bwd(x, weight, dy, bias=None, init_state=None, d_final=None, *,
                          activation: bool = True, out=None, workspace=None, stream=None) -> dict:
    """Gradients of ssd_causal_conv1d: of sum(dy * y) + sum(d_final * final_state).
    x, dy [b,L,C] in one dtype; weight [C,K], bias [C], init_state and d_final
    [b,C,K-1] float32 (the last three optional).  Returns a dict dx (x's dtype),
    dweight [C,K], dbias [C], d_init [b,C,K-1] (float32); ``out`` may hold
    preallocated tensors under the same keys; dx must not overlap x or dy."""
    entry = _entry("ssd_causal_conv1d_bwd", SsdConv1dBwdArgs)
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    b, L, Cn = shape
    K = weight.shape[1]
    state = (b, Cn, K - 1)
    ins = (_addr(x, "x", shape, dt, dev), _addr(weight, "weight", (Cn, K), _F32, dev),
           0 if bias is None else _addr(bias, "bias", (Cn,), _F32, dev),
           0 if init_state is None or K == 1 else _addr(init_state, "init_state", state, _F32, dev),
           _addr(dy, "dy", shape, dt, dev),
           0 if d_final is None or K == 1 else _addr(d_final, "d_final", state, _F32, dev))
    need = ssd_causal_conv1d_bwd_workspace_size(b, L, Cn, K, dt)
    if need == 0:
        raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_causal_conv1d_bwd (sizes)")
    o = dict(out) if out else {}
    outs = []
    for name, shp, dtype in (("dx", shape, dt), ("dweight", (Cn, K), _F32), ("dbias", (Cn,), _F32),
                             ("d_init", state, _F32)):
        o[name], p = _output(o.get(name), name, shp, dtype, x, dev, stream)
        outs.append(p)
    if K == 1:
        outs[3] = 0
    ws, size, keep = _workspace(workspace, need, x, dev, stream)
    _call(entry, stream, dev, b, L, Cn, K, _dtype_code(x), 1 if activation else 0, *ins, *outs, ws, size)
    return o


def ssd_gated_scan(x, gate_a, gate_x, decay, init_state=None, reset=None, *, scale: float = 8.0,
                   y=None, final_state=None, return_final_state: bool = False, states=None,
                   return_states: bool = False, stream=None):
    """The gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2)
    sigma(gate_x_t) x_t with log a_t = -scale softplus(decay) sigma(gate_a_t);
    y_t = h_t.  x, gate_a, gate_x [b,L,C] in one dtype; decay [C] and init_state
    [b,C] float32; reset [b,L] bool or uint8, nonzero where a token starts a new
    sequence.  Returns y, then the final state [b,C] and the states entering
    every 64th token [b,ceil(L/64),C] (for ssd_gated_scan_bwd), each when asked
    for or given.  Outputs must not overlap inputs."""
    entry = _entry("ssd_gated_scan", SsdGatedScanArgs)
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    b, L, Cn = shape
    state, kept = (b, Cn), (b, -(-L // SSD_GATED_SCAN_INTERVAL), Cn)
    y, yp = _output(y, "y", shape, dt, x, dev, stream)
    fp = sp = 0
    if final_state is not None or return_final_state:
        final_state, fp = _output(final_state, "final_state", state, _F32, x, dev, stream)
    if states is not None or return_states:
        states, sp = _output(states, "states", kept, _F32, x, dev, stream)
    _call(entry, stream, dev, b, L, Cn, _dtype_code(x), scale, _addr(x, "x", shape, dt, dev),
          _addr(gate_a, "gate_a", shape, dt, dev), _addr(gate_x, "gate_x", shape, dt, dev),
          _addr(decay, "decay", (Cn,), _F32, dev), _reset_addr(reset, (b, L), dev),
          0 if init_state is None else _addr(init_state, "init_state", state, _F32, dev),
          yp, fp, sp)
    if final_state is None and states is None:
        return y
    return (y,) + tuple(t for t in (final_state, states) if t is not None)


def ssd_gated_scan_check_status(stream=None) -> int:
    """Synchronises the stream; SSD_ERR_TIMEOUT if a ssd_gated_scan or
    ssd_gated_scan_bwd on this device gave up on an internal wait since the last
    check, else 0."""
    return int(load_library().ssd_gated_scan_check_status(_stream_ptr(stream)))


@functools.lru_cache(maxsize=1024)
def ssd_gated_scan_bwd_workspace_size(batch, seqlen, channels, dtype=torch.bfloat16) -> int:
    a = SsdGatedScanBwdArgs(batch=batch, seqlen=seqlen, channels=channels, scale=1.0,
                            dtype=SSD_BF16 if dtype == torch.bfloat16 else SSD_F32)
    return int(load_library().ssd_gated_scan_bwd_workspace_size(ctypes.byref(a)))


def ssd_gated_scan_bwd(x, gate_a, gate_x, decay, dy, states, reset=None, d_final=None, *,
                       scale: float = 8.0, out=None, workspace=None, stream=None) -> dict:
    """Gradients of ssd_gated_scan: of sum(dy * y) + sum(d_final * final_state).
    ``states`` is what the forward returned with return_states for the same
    inputs.  Returns a dict dx, dgate_a, dgate_x (x's dtype), ddecay [C] and
    d_init [b,C] (float32); ``out`` may hold preallocated tensors under the same
    keys, which must not overlap inputs."""
    entry = _entry("ssd_gated_scan_bwd", SsdGatedScanBwdArgs)
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    b, L, Cn = shape
    state, kept = (b, Cn), (b, -(-L // SSD_GATED_SCAN_INTERVAL), Cn)
    ins = (_addr(x, "x", shape, dt, dev), _addr(gate_a, "gate_a", shape, dt, dev),
           _addr(gate_x, "gate_x", shape, dt, dev), _addr(decay, "decay", (Cn,), _F32, dev),
           _reset_addr(reset, (b, L), dev), _addr(states, "states", kept, _F32, dev),
           _addr(dy, "dy", shape, dt, dev),
           0 if d_final is None else _addr(d_final, "d_final", state, _F32, dev))
    need = ssd_gated_scan_bwd_workspace_size(b, L, Cn, dt)
    if need == 0:
        raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_gated_scan_bwd (sizes)")
    o = dict(out) if out else {}
    outs = []
    for name, shp, dtype in (("dx", shape, dt), ("dgate_a", shape, dt), ("dgate_x", shape, dt),
                             ("ddecay", (Cn,), _F32), ("d_init", state, _F32)):
        o[name], p = _output(o.get(name), name, shp, dtype, x, dev, stream)
        outs.append(p)
    ws, size, keep = _workspace(workspace, need, x, dev, stream)
    _call(entry, stream, dev, b, L, Cn, _dtype_code(x), scale, *ins, *outs, ws, size)
    return o


def ssd_gated_state_update(state, x, gate_a, gate_x, decay, reset=None, *, scale: float = 8.0,
                           y=None, new_state=None, stream=None):
    """One decode step of the gated linear recurrence: x, gate_a, gate_x [b,C] in
    one dtype, decay [C] and state [b,C] float32, reset [b] bool or uint8.  The
    state is updated in place unless ``new_state`` is given, which then receives
    it.  Returns y [b,C]."""
    entry = _entry("ssd_gated_state_update", SsdGatedStateUpdateArgs)
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    b, Cn = shape
    y, yp = _output(y, "y", shape, dt, x, dev, stream)
    sp = _addr(state, "state", shape, _F32, dev)
    _call(entry, stream, dev, b, Cn, _dtype_code(x), scale, sp, _addr(x, "x", shape, dt, dev),
          _addr(gate_a, "gate_a", shape, dt, dev), _addr(gate_x, "gate_x", shape, dt, dev),
          _addr(decay, "decay", (Cn,), _F32, dev), _reset_addr(reset, (b,), dev),
          sp if new_state is None else _addr(new_state, "new_state", shape, _F32, dev), yp)
    return y


def _head_rows(t, name, shape, dtype, dev):
    """(address, elements between tokens) of t [b,L,H,D], whose heads are dense
    within a token and whose tokens are evenly spaced (a slice of packed rows)."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be {dtype} and on the device of the other tensors")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    b, L, H, D = shape
    sb, sl, sh, sd = t.stride()
    if sd != 1 or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a token must be dense")
    if L > 1 and b > 1 and sb != L * sl:
        raise ValueError(f"{name}: the tokens of all batch rows must be evenly spaced")
    return t.data_ptr(), (sl if L > 1 else sb if b > 1 else H * D)


def _head_output(given, name, shape, dtype, like, dev, stream):
    if given is None:
        t = _empty(shape, dtype, like, stream)
        return t, t.data_ptr(), shape[2] * shape[3]
    return (given, *_head_rows(given, name, shape, dtype, dev))


def _rotation(q, q_weight, k_weight, inv_freq, positions, dev):
    """Addresses of the weights, frequencies and positions, and rot_dim."""
    b, L, _, D = q.shape
    n = 0 if inv_freq is None else inv_freq.numel()
    return (0 if q_weight is None else _addr(q_weight, "q_weight", (D,), _F32, dev),
            0 if k_weight is None else _addr(k_weight, "k_weight", (D,), _F32, dev),
            0 if n == 0 else _addr(inv_freq, "inv_freq", (n,), _F32, dev),
            0 if positions is None else _addr(positions, "positions", (b, L), torch.int64, dev)), 2 * n


def _key_shape(q, k):
    b, L, _, D = q.shape
    return (b, L, k.shape[2], D)


def ssd_qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions=None, *, eps: float = 1e-5,
                     adjacent: bool = False, q_out=None, k_out=None, stream=None):
    """RMSNorm over each head of the queries and keys (C and B in the scan's dual
    form) and, in the same pass, the rotation of each head's first
    2 * len(inv_freq) elements by position * inv_freq: pairs (j, j + len) or,
    with ``adjacent``, (2j, 2j + 1).  q [b,L,Hq,D], k [b,L,Hk,D] (or None) in one
    dtype, each possibly a slice of packed rows (heads dense within a token,
    tokens evenly spaced); q_weight, k_weight [D] float32 or None; inv_freq
    float32 or None (no rotation); positions [b,L] int64 or None (0, 1, ... in
    each row).  q_out / k_out may be q / k (in place) or such slices.  Returns
    (q_out, k_out)."""
    entry = _entry("ssd_qk_norm_rope", SsdQkNormRopeArgs)
    qs, dt, dev = q.shape, q.dtype, q.get_device()
    b, L, hq, D = qs
    qp, q_stride = _head_rows(q, "q", qs, dt, dev)
    q_out, qo, qo_stride = _head_output(q_out, "q_out", qs, dt, q, dev, stream)
    hk = kp = ko = k_stride = ko_stride = 0
    if k is not None:
        ks = _key_shape(q, k)
        hk = ks[2]
        kp, k_stride = _head_rows(k, "k", ks, dt, dev)
        k_out, ko, ko_stride = _head_output(k_out, "k_out", ks, dt, q, dev, stream)
    ptrs, rot = _rotation(q, q_weight, k_weight, inv_freq, positions, dev)
    _call(entry, stream, dev, b, L, hq, hk, D, rot, q_stride, k_stride, qo_stride, ko_stride, _dtype_code(q),
          1 if adjacent else 0, eps, qp, kp, *ptrs, qo, ko)
    return q_out, (k_out if k is not None else None)


@functools.lru_cache(maxsize=1024)
def ssd_qk_norm_rope_bwd_workspace_size(batch, seqlen, q_heads, k_heads, headdim, rot_dim,
                                        dtype=torch.bfloat16) -> int:
    a = SsdQkNormRopeBwdArgs(batch=batch, seqlen=seqlen, q_heads=q_heads, k_heads=k_heads,
                             headdim=headdim, rot_dim=rot_dim,
                             dtype=SSD_BF16 if dtype == torch.bfloat16 else SSD_F32)
    return int(load_library().ssd_qk_norm_rope_bwd_workspace_size(ctypes.byref(a)))


def ssd_qk_norm_rope_bwd(q, k, q_weight, k_weight, inv_freq, dq_out, dk_out, positions=None, *,
                         eps: float = 1e-5, adjacent: bool = False, out=None, workspace=None,
                         stream=None) -> dict:
    """Gradients of ssd_qk_norm_rope from those of its outputs (dq_out, dk_out: q's
    and k's shapes, dense or slices as there).  Returns a dict dq, dk (q's dtype;
    dk absent without k), dq_weight, dk_weight [D] (float32); ``out`` may hold
    preallocated tensors under the same keys, dq and dk also as slices of packed
    rows; they must not overlap inputs."""
    entry = _entry("ssd_qk_norm_rope_bwd", SsdQkNormRopeBwdArgs)
    qs, dt, dev = q.shape, q.dtype, q.get_device()
    b, L, hq, D = qs
    o = dict(out) if out else {}

    def side(name, t, d_out, shape):
        """input, incoming gradient, outgoing gradient (address, stride), weight's gradient"""
        g, w = "d" + name, f"d{name}_weight"
        ins = _head_rows(t, name, shape, dt, dev) + _head_rows(d_out, g + "_out", shape, dt, dev)
        o[g], gp, stride = _head_output(o.get(g), g, shape, dt, q, dev, stream)
        o[w], wp = _output(o.get(w), w, (D,), _F32, q, dev, stream)
        return (*ins, gp, stride, wp)

    ptrs, rot = _rotation(q, q_weight, k_weight, inv_freq, positions, dev)
    hk = 0 if k is None else k.shape[2]
    need = ssd_qk_norm_rope_bwd_workspace_size(b, L, hq, hk, D, rot, dt)
    if need == 0:
        raise SsdError(SSD_ERR_UNSUPPORTED, "ssd_qk_norm_rope_bwd (sizes)")
    qp, q_stride, qg, qg_stride, dq, dq_stride, dqw = side("q", q, dq_out, qs)
    kp = k_stride = kg = kg_stride = dk = dk_stride = dkw = 0
    if k is not None:
        kp, k_stride, kg, kg_stride, dk, dk_stride, dkw = side("k", k, dk_out, _key_shape(q, k))
    ws, size, keep = _workspace(workspace, need, q, dev, stream)
    _call(entry, stream, dev, b, L, hq, hk, D, rot, q_stride, k_stride, qg_stride, kg_stride, dq_stride, dk_stride,
          _dtype_code(q), 1 if adjacent else 0, eps, qp, kp, *ptrs, qg, kg, dq, dk, dqw, dkw, ws, size)
    return o
