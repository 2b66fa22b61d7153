"""Thin Python binding of libssmscan.so (include/ssmscan.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their data pointers and the current CUDA stream are passed to the
C ABI, and a non-OK status becomes an ``SsmError``.  Outputs (and the
workspace the library asks for) are allocated here with torch when the caller
does not pass them; every step of the computation runs in the library's
kernels.  Importing this module fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# SSM_DEBUG_BOUNDS=1 selects the debug-bounds build (every kernel checks its
# global indices and records misses for check_device_errors)
DEBUG_BOUNDS = os.environ.get("SSM_DEBUG_BOUNDS", "") == "1"
LIB_PATH = os.path.join(_PKG, "libssmscan_debug.so" if DEBUG_BOUNDS else "libssmscan.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "ssmscan.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m selective_state_space_25_b200.build` "
        "(the CUDA path has no fallback)")

_lib = ctypes.CDLL(LIB_PATH)

SSM_OK, SSM_ERR_INVALID_ARG, SSM_ERR_UNSUPPORTED, SSM_ERR_WORKSPACE, SSM_ERR_CUDA, \
    SSM_ERR_DEVICE_TIMEOUT, SSM_ERR_DEVICE_BOUNDS = range(7)
SSM_F32, SSM_BF16 = 0, 1
_STATUS = {0: "SSM_OK", 1: "SSM_ERR_INVALID_ARG", 2: "SSM_ERR_UNSUPPORTED", 3: "SSM_ERR_WORKSPACE",
           4: "SSM_ERR_CUDA", 5: "SSM_ERR_DEVICE_TIMEOUT", 6: "SSM_ERR_DEVICE_BOUNDS"}

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t
_NO_SIZE = _SZ(-1).value  # a size query's answer for invalid sizes

_lib.ssm_last_error.restype = ctypes.c_char_p
_lib.ssm_version.restype = ctypes.c_char_p
_lib.ssm_scan_fwd_workspace_bytes.argtypes = [_I64] * 4
_lib.ssm_scan_fwd_workspace_bytes.restype = _SZ
_lib.ssm_scan_fwd.argtypes = [_P] * 8 + [_INT, _P, _P, _P] + [_I64] * 4 + [_INT, _P, _SZ, _P]
_lib.ssm_scan_fwd.restype = _INT
_lib.ssm_scan_bwd_workspace_bytes.argtypes = [_I64] * 4
_lib.ssm_scan_bwd_workspace_bytes.restype = _SZ
_lib.ssm_scan_bwd_fast_workspace_bytes.argtypes = [_I64] * 4
_lib.ssm_scan_bwd_fast_workspace_bytes.restype = _SZ
_lib.ssm_scan_bwd_saved_workspace_bytes.argtypes = [_I64] * 4
_lib.ssm_scan_bwd_saved_workspace_bytes.restype = _SZ
_lib.ssm_scan_bwd.argtypes = [_P] * 8 + [_INT] + [_P] * 12 + [_I64] * 4 + [_INT, _P, _SZ, _P]
_lib.ssm_scan_bwd.restype = _INT
_lib.ssm_scan_fwd_save.argtypes = [_P] * 8 + [_INT, _P, _P, _P, _P, _SZ] + [_I64] * 4 + [_INT, _P]
_lib.ssm_scan_fwd_save.restype = _INT
_lib.ssm_scan_fwd_save_ex.argtypes = _lib.ssm_scan_fwd_save.argtypes[:-1] + [_P, _SZ, _P]
_lib.ssm_scan_fwd_save_ex.restype = _INT
_lib.ssm_scan_bwd_saved.argtypes = ([_P] * 8 + [_INT] + [_P] * 11 + [_I64] * 4
                                    + [_INT, _P, _SZ, _P])
_lib.ssm_scan_bwd_saved.restype = _INT
_lib.ssm_scan_bwd_saved_ex.argtypes = (_lib.ssm_scan_bwd_saved.argtypes[:-1]
                                       + [_P, _SZ, _P])
_lib.ssm_scan_bwd_saved_ex.restype = _INT
_lib.ss2d_scan_fwd_workspace_bytes.argtypes = [_I64] * 5
_lib.ss2d_scan_fwd_workspace_bytes.restype = _SZ
_lib.ss2d_scan_fwd_fast_workspace_bytes.argtypes = [_I64] * 5
_lib.ss2d_scan_fwd_fast_workspace_bytes.restype = _SZ
_lib.ss2d_scan_fwd.argtypes = [_P] * 7 + [_INT, _P] + [_I64] * 5 + [_INT, _P, _SZ, _P]
_lib.ss2d_scan_fwd.restype = _INT
_lib.ssm_state_update.argtypes = [_P] * 9 + [_INT, _P] + [_I64] * 3 + [_INT, _P]
_lib.ssm_state_update.restype = _INT
_lib.ssm_conv_state_update.argtypes = [_P, _P, _P, _I64] + [_P] * 9 + [_INT, _P] + [_I64] * 3 + [_INT, _P]
_lib.ssm_conv_state_update.restype = _INT
_lib.ss2d_cross_scan.argtypes = [_P, _P] + [_I64] * 4 + [_INT, _P]
_lib.ss2d_cross_scan.restype = _INT
_lib.ss2d_cross_merge.argtypes = [_P, _P] + [_I64] * 4 + [_INT, _P]
_lib.ss2d_cross_merge.restype = _INT
_lib.ss2d_scan_fwd_ex.argtypes = [_P] * 7 + [_INT, _P] + [_I64] * 5 + [_INT, _INT, _P, _SZ, _P]
_lib.ss2d_scan_fwd_ex.restype = _INT
_lib.ss2d_cross_scan_ex.argtypes = [_P, _P] + [_I64] * 4 + [_INT, _INT, _P]
_lib.ss2d_cross_scan_ex.restype = _INT
_lib.ss2d_cross_merge_ex.argtypes = [_P, _P] + [_I64] * 4 + [_INT, _INT, _P]
_lib.ss2d_cross_merge_ex.restype = _INT
SS2D_ORDERS = {"cross": 0, "snake": 1}
_ROWS = [_P, _I64]  # an activation and its row stride
_lib.ssm_gated_scan_states_bytes.argtypes = [_I64] * 3
_lib.ssm_gated_scan_states_bytes.restype = _SZ
_lib.ssm_gated_scan_fwd.argtypes = (_ROWS * 3 + [_P] * 3 + _ROWS + [_P] * 3 + _ROWS + [_P, _SZ]
                                    + [_I64] * 3 + [_INT, _P])
_lib.ssm_gated_scan_fwd.restype = _INT
_lib.ssm_gated_scan_bwd_workspace_bytes.argtypes = [_I64] * 3
_lib.ssm_gated_scan_bwd_workspace_bytes.restype = _SZ
_lib.ssm_gated_scan_bwd.argtypes = (_ROWS * 3 + [_P] * 3 + _ROWS + [_P] + _ROWS + [_P] + _ROWS * 4
                                    + [_P] * 4 + [_I64] * 3 + [_INT, _P, _SZ, _P, _SZ, _P])
_lib.ssm_gated_scan_bwd.restype = _INT
_lib.ssm_gated_state_update.argtypes = ([_P] + _ROWS * 3 + [_P] * 3 + _ROWS * 2 + [_I64] * 2
                                        + [_INT, _P])
_lib.ssm_gated_state_update.restype = _INT
_lib.ssm_conv1d_fwd.argtypes = (_ROWS + [_P, _P, _INT] + [_P] * 3 + _ROWS + [_I64] * 4 + [_INT, _P])
_lib.ssm_conv1d_fwd.restype = _INT
_lib.ssm_conv1d_bwd_workspace_bytes.argtypes = [_I64] * 4
_lib.ssm_conv1d_bwd_workspace_bytes.restype = _SZ
_lib.ssm_conv1d_bwd.argtypes = (_ROWS + [_P, _P, _INT] + [_P] * 2 + _ROWS * 2 + [_P] * 2 + [_I64] * 4
                                + [_INT, _P, _SZ, _P])
_lib.ssm_conv1d_bwd.restype = _INT
_lib.ssm_conv1d_update.argtypes = [_P] + _ROWS + [_P, _P, _INT] + _ROWS + [_I64] * 3 + [_INT, _P]
_lib.ssm_conv1d_update.restype = _INT
_F32 = ctypes.c_float
_lib.ssm_gated_norm_fwd.argtypes = (_ROWS * 2 + [_P, _I64, _F32, _INT] + _ROWS + [_I64] * 2
                                    + [_INT, _P])
_lib.ssm_gated_norm_fwd.restype = _INT
_lib.ssm_gated_norm_bwd_workspace_bytes.argtypes = [_I64] * 3
_lib.ssm_gated_norm_bwd_workspace_bytes.restype = _SZ
_lib.ssm_gated_norm_bwd.argtypes = (_ROWS * 2 + [_P, _I64, _F32, _INT] + _ROWS * 3 + [_P]
                                    + [_I64] * 2 + [_INT, _P, _SZ, _P])
_lib.ssm_gated_norm_bwd.restype = _INT
_lib.ssm_add_norm_fwd.argtypes = (_ROWS * 2 + [_P] * 3 + [_F32] + _ROWS * 2 + [_I64] * 2
                                  + [_INT, _INT, _P])
_lib.ssm_add_norm_fwd.restype = _INT
_lib.ssm_add_norm_bwd_workspace_bytes.argtypes = [_I64] * 2
_lib.ssm_add_norm_bwd_workspace_bytes.restype = _SZ
_lib.ssm_add_norm_bwd.argtypes = (_ROWS * 2 + [_P] * 3 + [_F32] + _ROWS * 4 + [_P] * 3 + [_I64] * 2
                                  + [_INT, _INT, _P, _SZ, _P])
_lib.ssm_add_norm_bwd.restype = _INT
_lib.ssm_check_device_errors.argtypes = [_P]
_lib.ssm_check_device_errors.restype = _INT
_lib.ssm_debug_bounds_enabled.argtypes = []
_lib.ssm_debug_bounds_enabled.restype = _INT
_lib.ssm_debug_bounds_self_test.argtypes = [_P]
_lib.ssm_debug_bounds_self_test.restype = _INT


class SsmError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libssmscan.so (for tests that call the C ABI directly)."""
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/ssmscan.h declares."""
    text = open(HEADER, encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ssm_\w+|ss2d_\w+)\s*\(", text)))


def version() -> str:
    return _lib.ssm_version().decode()


def last_error() -> str:
    return _lib.ssm_last_error().decode()


def _check(status: int, where: str) -> None:
    if status != SSM_OK:
        raise SsmError(status, where, last_error())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    if t.dtype == torch.float32:
        return SSM_F32
    raise TypeError(f"unsupported activation dtype {t.dtype} (bf16 or fp32)")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, shape, dtype, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def ssm_scan_fwd_workspace_bytes(b: int, L: int, d_in: int, d_state: int) -> int:
    return int(_lib.ssm_scan_fwd_workspace_bytes(b, L, d_in, d_state))


def ssm_scan_fwd(u, delta, A, B, C, D=None, z=None, dt_bias=None, delta_softplus=True,
                 h0=None, h_last=None, y=None, workspace=None, stream=None, chunk_states=None):
    """Selective scan forward (see include/ssmscan.h).  u, delta, z: (b, L, d_in);
    A: (d_in, N) fp32; B, C: (b, L, N); D, dt_bias: (d_in,) fp32; h0, h_last:
    (b, d_in, N) fp32.  Returns y (b, L, d_in).  With ``chunk_states`` (a
    device buffer of ssm_scan_bwd_workspace_bytes(...) bytes) the forward
    also saves the chunk-start states for ssm_scan_bwd(..., states=...).
    Unless ``workspace`` is given, the split scan's workspace
    (ssm_scan_fwd_workspace_bytes) is allocated when it is not 0."""
    if u.dim() != 3:
        raise ValueError("u must be (b, L, d_in)")
    b, L, d_in = u.shape
    N = A.shape[-1]
    dev, act = u.device, u.dtype
    f32 = torch.float32
    _need(u, "u", (b, L, d_in), act, dev)
    _need(delta, "delta", (b, L, d_in), act, dev)
    _need(A, "A", (d_in, N), f32, dev)
    _need(B, "B", (b, L, N), act, dev)
    _need(C, "C", (b, L, N), act, dev)
    _need(D, "D", (d_in,), f32, dev)
    _need(z, "z", (b, L, d_in), act, dev)
    _need(dt_bias, "dt_bias", (d_in,), f32, dev)
    _need(h0, "h0", (b, d_in, N), f32, dev)
    _need(h_last, "h_last", (b, d_in, N), f32, dev)
    if y is None:
        y = torch.empty_like(u)
    _need(y, "y", (b, L, d_in), act, dev)
    ws_bytes = ssm_scan_fwd_workspace_bytes(b, L, d_in, N)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if chunk_states is not None:
        st = _lib.ssm_scan_fwd_save_ex(
            _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias),
            int(bool(delta_softplus)), _ptr(h0), _ptr(h_last), _ptr(y), _ptr(chunk_states),
            chunk_states.numel() * chunk_states.element_size(), b, L, d_in, N, _dtype_code(u),
            _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
            _stream(stream))
        _check(st, "ssm_scan_fwd_save")
        return y
    st = _lib.ssm_scan_fwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                           _ptr(dt_bias), int(bool(delta_softplus)), _ptr(h0), _ptr(h_last),
                           _ptr(y), b, L, d_in, N, _dtype_code(u), _ptr(workspace),
                           0 if workspace is None else workspace.numel() * workspace.element_size(),
                           _stream(stream))
    _check(st, "ssm_scan_fwd")
    return y


def ssm_scan_bwd_workspace_bytes(b: int, L: int, d_in: int, d_state: int) -> int:
    return int(_lib.ssm_scan_bwd_workspace_bytes(b, L, d_in, d_state))


def ssm_scan_bwd_fast_workspace_bytes(b: int, L: int, d_in: int, d_state: int) -> int:
    return int(_lib.ssm_scan_bwd_fast_workspace_bytes(b, L, d_in, d_state))


def ssm_scan_bwd_saved_workspace_bytes(b: int, L: int, d_in: int, d_state: int) -> int:
    return int(_lib.ssm_scan_bwd_saved_workspace_bytes(b, L, d_in, d_state))


def ssm_scan_bwd(u, delta, A, B, C, dout, D=None, z=None, dt_bias=None, delta_softplus=True,
                 h0=None, dh_last=None, want_dh0=False, workspace=None, stream=None, out=None,
                 states=None):
    """Gradients of sum(dout * y) [+ sum(dh_last * h_last)] for ssm_scan_fwd
    with the same inputs.  Returns a dict: du, ddelta, dz (activation dtype,
    (b, L, d_in); dz only with z); dA (d_in, N), dB, dC (b, L, N), dD,
    ddt_bias (d_in) in fp32; dh0 (b, d_in, N) fp32 when want_dh0.  ``out``
    (a dict returned by an earlier call with the same shapes) is refilled
    in place instead of allocating.  ``states``: the chunk_states buffer a
    forward with the same inputs filled (ssm_scan_fwd(..., chunk_states=));
    the backward then starts from it (ssm_scan_bwd_saved_ex, with ``workspace``
    or an allocated one for its split when channels are few) and h0 is unused."""
    b, L, d_in = u.shape
    N = A.shape[1]
    dev, act, f32 = u.device, u.dtype, torch.float32
    _need(u, "u", (b, L, d_in), act, dev)
    _need(delta, "delta", (b, L, d_in), act, dev)
    _need(A, "A", (d_in, N), f32, dev)
    _need(B, "B", (b, L, N), act, dev)
    _need(C, "C", (b, L, N), act, dev)
    _need(dout, "dout", (b, L, d_in), act, dev)
    _need(D, "D", (d_in,), f32, dev)
    _need(z, "z", (b, L, d_in), act, dev)
    _need(dt_bias, "dt_bias", (d_in,), f32, dev)
    _need(h0, "h0", (b, d_in, N), f32, dev)
    _need(dh_last, "dh_last", (b, d_in, N), f32, dev)
    if out is not None:
        g = {k: out.get(k) for k in ("du", "ddelta", "dz", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")}
        for k, shp, dt in (("du", (b, L, d_in), act), ("ddelta", (b, L, d_in), act),
                           ("dz", (b, L, d_in), act), ("dA", (d_in, N), f32),
                           ("dB", (b, L, N), f32), ("dC", (b, L, N), f32), ("dD", (d_in,), f32),
                           ("ddt_bias", (d_in,), f32), ("dh0", (b, d_in, N), f32)):
            _need(g[k], k, shp, dt, dev)
    else:
        g = dict(du=torch.empty_like(u), ddelta=torch.empty_like(u),
                 dz=torch.empty_like(u) if z is not None else None,
                 dA=torch.empty((d_in, N), dtype=f32, device=dev),
                 dB=torch.empty((b, L, N), dtype=f32, device=dev),
                 dC=torch.empty((b, L, N), dtype=f32, device=dev),
                 dD=torch.empty(d_in, dtype=f32, device=dev),
                 ddt_bias=torch.empty(d_in, dtype=f32, device=dev),
                 dh0=torch.empty((b, d_in, N), dtype=f32, device=dev) if want_dh0 else None)
    if states is not None:
        aux = ssm_scan_bwd_saved_workspace_bytes(b, L, d_in, N)
        if workspace is None and 0 < aux < _NO_SIZE:  # else the call says what it refuses
            workspace = torch.empty(aux, dtype=torch.uint8, device=dev)
        st = _lib.ssm_scan_bwd_saved_ex(
            _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias),
            int(bool(delta_softplus)), _ptr(dout), _ptr(dh_last), _ptr(g["du"]),
            _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
            _ptr(g["dz"]), _ptr(g["ddt_bias"]), _ptr(g["dh0"]), b, L, d_in, N, _dtype_code(u),
            _ptr(states), states.numel() * states.element_size(), _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            _stream(stream))
        _check(st, "ssm_scan_bwd_saved")
        return {k: v for k, v in g.items() if v is not None}
    need = ssm_scan_bwd_fast_workspace_bytes(b, L, d_in, N)  # the fastest path's
    if workspace is None and need < _NO_SIZE:  # else the call says what it refuses
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _lib.ssm_scan_bwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                           _ptr(dt_bias), int(bool(delta_softplus)), _ptr(h0), _ptr(dout),
                           _ptr(dh_last), _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dA"]),
                           _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dz"]),
                           _ptr(g["ddt_bias"]), _ptr(g["dh0"]), b, L, d_in, N, _dtype_code(u),
                           _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "ssm_scan_bwd")
    return {k: v for k, v in g.items() if v is not None}


def ss2d_scan_fwd_workspace_bytes(b: int, H: int, W: int, d_in: int, d_state: int) -> int:
    return int(_lib.ss2d_scan_fwd_workspace_bytes(b, H, W, d_in, d_state))


def ss2d_scan_fwd_fast_workspace_bytes(b: int, H: int, W: int, d_in: int, d_state: int) -> int:
    return int(_lib.ss2d_scan_fwd_fast_workspace_bytes(b, H, W, d_in, d_state))


def ss2d_scan_fwd(u, delta, A, B, C, H, W, D=None, dt_bias=None, delta_softplus=True, y=None,
                  workspace=None, stream=None, order="cross"):
    """SS2D forward.  u: (b, H W, d_in); delta: (b, 4, H W, d_in); A: (4 d_in, N)
    fp32; B, C: (b, 4, H W, N); D, dt_bias: (4 d_in,) fp32; order "cross" or
    "snake".  Returns y (b, H W, d_in).  Without a ``workspace`` the binding
    allocates the one that lets the call take its fastest path."""
    b, L, d_in = u.shape
    N = A.shape[-1]
    if L != H * W:
        raise ValueError("u.shape[1] must be H*W")
    dev, act, f32 = u.device, u.dtype, torch.float32
    _need(delta, "delta", (b, 4, L, d_in), act, dev)
    _need(A, "A", (4 * d_in, N), f32, dev)
    _need(B, "B", (b, 4, L, N), act, dev)
    _need(C, "C", (b, 4, L, N), act, dev)
    _need(D, "D", (4 * d_in,), f32, dev)
    _need(dt_bias, "dt_bias", (4 * d_in,), f32, dev)
    _need(u, "u", (b, L, d_in), act, dev)
    if y is None:
        y = torch.empty_like(u)
    _need(y, "y", (b, L, d_in), act, dev)
    ws_bytes = ss2d_scan_fwd_fast_workspace_bytes(b, H, W, d_in, N)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = _lib.ss2d_scan_fwd_ex(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                               _ptr(dt_bias), int(bool(delta_softplus)), _ptr(y), b, H, W, d_in, N,
                               SS2D_ORDERS[order], _dtype_code(u), _ptr(workspace),
                            0 if workspace is None else workspace.numel() * workspace.element_size(),
                            _stream(stream))
    _check(st, "ss2d_scan_fwd")
    return y


def ssm_state_update(ssm_state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True,
                     y=None, stream=None):
    """One decode step; ssm_state (b, d_in, N) fp32 is updated in place.
    x, dt, z: (b, d_in); B, C: (b, N).  Returns y (b, d_in)."""
    b, d_in, N = ssm_state.shape
    dev, act, f32 = x.device, x.dtype, torch.float32
    _need(ssm_state, "ssm_state", (b, d_in, N), f32, dev)
    _need(x, "x", (b, d_in), act, dev)
    _need(dt, "dt", (b, d_in), act, dev)
    _need(A, "A", (d_in, N), f32, dev)
    _need(B, "B", (b, N), act, dev)
    _need(C, "C", (b, N), act, dev)
    _need(D, "D", (d_in,), f32, dev)
    _need(z, "z", (b, d_in), act, dev)
    _need(dt_bias, "dt_bias", (d_in,), f32, dev)
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", (b, d_in), act, dev)
    st = _lib.ssm_state_update(_ptr(ssm_state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                               _ptr(D), _ptr(z), _ptr(dt_bias), int(bool(dt_softplus)), _ptr(y),
                               b, d_in, N, _dtype_code(x), _stream(stream))
    _check(st, "ssm_state_update")
    return y


def ssm_conv_state_update(conv_state, conv_weight, ssm_state, x, dt, A, B, C, conv_bias=None,
                          D=None, z=None, dt_bias=None, dt_softplus=True, y=None, stream=None):
    """One decode step with the causal-conv1d step in front; conv_state
    (b, d_in, d_conv) in the activation dtype and ssm_state (b, d_in, N) fp32
    are updated in place.  conv_weight (d_in, d_conv) fp32.  Returns y (b, d_in)."""
    b, d_in, N = ssm_state.shape
    d_conv = conv_state.shape[-1]
    dev, act, f32 = x.device, x.dtype, torch.float32
    _need(conv_state, "conv_state", (b, d_in, d_conv), act, dev)
    _need(conv_weight, "conv_weight", (d_in, d_conv), f32, dev)
    _need(conv_bias, "conv_bias", (d_in,), f32, dev)
    _need(ssm_state, "ssm_state", (b, d_in, N), f32, dev)
    _need(x, "x", (b, d_in), act, dev)
    _need(dt, "dt", (b, d_in), act, dev)
    _need(A, "A", (d_in, N), f32, dev)
    _need(B, "B", (b, N), act, dev)
    _need(C, "C", (b, N), act, dev)
    _need(D, "D", (d_in,), f32, dev)
    _need(z, "z", (b, d_in), act, dev)
    _need(dt_bias, "dt_bias", (d_in,), f32, dev)
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", (b, d_in), act, dev)
    st = _lib.ssm_conv_state_update(_ptr(conv_state), _ptr(conv_weight), _ptr(conv_bias), d_conv,
                                    _ptr(ssm_state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                                    _ptr(D), _ptr(z), _ptr(dt_bias), int(bool(dt_softplus)),
                                    _ptr(y), b, d_in, N, _dtype_code(x), _stream(stream))
    _check(st, "ssm_conv_state_update")
    return y


def ss2d_cross_scan(u, H, W, xs=None, stream=None, order="cross"):
    """xs[b, k, l, d] = u[b, p_k(l), d]; u (b, H W, d_in) -> xs (b, 4, H W, d_in)."""
    b, L, d_in = u.shape
    if xs is None:
        xs = torch.empty((b, 4, L, d_in), dtype=u.dtype, device=u.device)
    _need(u, "u", (b, L, d_in), u.dtype, u.device)
    _need(xs, "xs", (b, 4, L, d_in), u.dtype, u.device)
    _check(_lib.ss2d_cross_scan_ex(_ptr(u), _ptr(xs), b, H, W, d_in, SS2D_ORDERS[order],
                                   _dtype_code(u), _stream(stream)), "ss2d_cross_scan")
    return xs


def ss2d_cross_merge(ys, H, W, y=None, stream=None, order="cross"):
    """y[b, p, d] = sum_k ys[b, k, l_k(p), d]; ys (b, 4, H W, d_in) -> y (b, H W, d_in)."""
    b, K, L, d_in = ys.shape
    if y is None:
        y = torch.empty((b, L, d_in), dtype=ys.dtype, device=ys.device)
    _need(ys, "ys", (b, 4, L, d_in), ys.dtype, ys.device)
    _need(y, "y", (b, L, d_in), ys.dtype, ys.device)
    _check(_lib.ss2d_cross_merge_ex(_ptr(ys), _ptr(y), b, H, W, d_in, SS2D_ORDERS[order],
                                    _dtype_code(ys), _stream(stream)), "ss2d_cross_merge")
    return y


# ------------------------------------------------- around the scan
# Activations of these calls may have strided rows: the last dimension
# adjacent, the leading ones collapsible to rows a fixed stride apart (a half of
# a projection's output).  The calls run on the inputs' device whatever the
# current one is; what they allocate comes from the pool of the stream they run
# on.

def _device_of(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a CUDA device")
    return t.device


def _rows(t, name, shape, dtype, device):
    """(pointer, row stride) of an activation; (None, 0) without one."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    d = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), d
    st = t.stride()
    if d > 1 and st[-1] != 1:
        raise ValueError(f"{name}: its last dimension must be adjacent")
    ld, span = None, None  # the rows' stride, from the innermost leading dimension longer than 1
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = span = s
        elif s != span:
            raise ValueError(f"{name}: its rows must be a fixed stride apart")
        span *= n
    if ld is None:
        ld = d
    if ld < d:
        raise ValueError(f"{name}: its rows overlap (stride {ld} for {d} elements)")
    return t.data_ptr(), ld


def _launch(fn, where, device, stream, *args):
    """Calls the library on `device` and `stream` (None: its current one)."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if device.index == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != SSM_OK:
        raise SsmError(status, where, last_error())


class _Pool:
    """Allocates on the stream a call runs on, so that memory the caching
    allocator hands out is not still in use on another one."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream
        if stream is not None and not hasattr(stream, "cuda_stream"):
            self.stream = torch.cuda.ExternalStream(int(stream), device=device)

    def like(self, t, dtype=None):
        """A contiguous tensor of t's shape (and type)."""
        if self.stream is None:
            return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)
        with torch.cuda.stream(self.stream):
            return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)

    def new(self, t, shape, dtype):
        """A tensor of this shape and type on t's device."""
        if self.stream is None:
            return t.new_empty(shape, dtype=dtype)
        with torch.cuda.stream(self.stream):
            return t.new_empty(shape, dtype=dtype)


def _workspace(workspace, nbytes, pool, ref):
    """(tensor, pointer, bytes) of the given workspace, or of one from the pool
    for the bytes the library asks for on its device; none for sizes that it
    refuses, which the call itself then says."""
    if workspace is None:
        if pool.device.index == torch._C._cuda_getDevice():
            n = nbytes()
        else:
            with torch.cuda.device(pool.device):
                n = nbytes()
        if n == _NO_SIZE:
            return None, None, 0
        workspace = pool.new(ref, max(int(n), 1), torch.uint8)
        return workspace, workspace.data_ptr(), int(n)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    if workspace.device != pool.device or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be contiguous on {pool.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def ssm_gated_scan_states_bytes(b: int, L: int, d_in: int) -> int:
    return int(_lib.ssm_gated_scan_states_bytes(b, L, d_in))


def ssm_gated_scan_bwd_workspace_bytes(b: int, L: int, d_in: int) -> int:
    return int(_lib.ssm_gated_scan_bwd_workspace_bytes(b, L, d_in))


def _gated_inputs(u, gate_a, gate_x, A, bias_a, bias_x, z, shape, dev):
    act, d = u.dtype, shape[-1]
    f32 = torch.float32
    _need(A, "A", (d,), f32, dev)
    _need(bias_a, "bias_a", (d,), f32, dev)
    _need(bias_x, "bias_x", (d,), f32, dev)
    return (*_rows(u, "u", shape, act, dev), *_rows(gate_a, "gate_a", shape, act, dev),
            *_rows(gate_x, "gate_x", shape, act, dev), _ptr(A), _ptr(bias_a), _ptr(bias_x),
            *_rows(z, "z", shape, act, dev))


def _chunk_states(states, name, b, L, d, dev):
    if states is None:
        return None, 0
    if not isinstance(states, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if states.device != dev or not states.is_contiguous():
        raise ValueError(f"{name}: must be contiguous on {dev}")
    return states.data_ptr(), states.numel() * states.element_size()


def ssm_gated_scan_fwd(u, gate_a, gate_x, A, bias_a=None, bias_x=None, z=None, seq_start=None,
                       h0=None, h_last=None, y=None, chunk_states=None, stream=None):
    """Gated linear recurrence (see include/ssmscan.h).  u, gate_a, gate_x, z:
    (b, L, d_in); A, bias_a, bias_x: (d_in,) fp32; seq_start: (b, L) uint8;
    h0, h_last: (b, d_in) fp32.  Returns y (b, L, d_in).  With
    ``chunk_states`` (a device buffer of ssm_gated_scan_states_bytes(...)
    bytes) the states that ssm_gated_scan_bwd starts from are kept."""
    dev = _device_of(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be (b, L, d_in)")
    shape = u.shape
    b, L, d = shape
    code = _dtype_code(u)
    ins = _gated_inputs(u, gate_a, gate_x, A, bias_a, bias_x, z, shape, dev)
    _need(seq_start, "seq_start", (b, L), torch.uint8, dev)
    _need(h0, "h0", (b, d), torch.float32, dev)
    _need(h_last, "h_last", (b, d), torch.float32, dev)
    states = _chunk_states(chunk_states, "chunk_states", b, L, d, dev)
    if y is None:
        y = _Pool(dev, stream).like(u)
    _launch(_lib.ssm_gated_scan_fwd, "ssm_gated_scan_fwd", dev, stream, *ins, _ptr(seq_start),
            _ptr(h0), _ptr(h_last), *_rows(y, "y", shape, u.dtype, dev), *states, b, L, d, code)
    return y


def _outputs(out, likes, params, pool, dev):
    """The outputs {name: tensor}, from ``out`` where it has them, else new: likes
    {name: a tensor of its shape and type, as contiguous rows}, params {name: the
    fp32 parameter it is the gradient of}."""
    if out is None:
        got = {k: pool.like(t) for k, t in likes.items()}
        if len(params) > 1 and len({t.shape for t in params.values()}) == 1:
            ref = next(iter(params.values()))  # one allocation, a row for each
            got.update(zip(params, pool.new(ref, (len(params), *ref.shape), torch.float32).unbind(0)))
        else:
            got.update((k, pool.like(t)) for k, t in params.items())
        return got
    got = {k: pool.like(t) if out.get(k) is None else out[k] for k, t in likes.items()}
    for k, t in params.items():
        g = out.get(k)
        if g is not None:
            _need(g, k, t.shape, torch.float32, dev)
        got[k] = pool.like(t) if g is None else g
    return got


def ssm_gated_scan_bwd(u, gate_a, gate_x, A, dout, states, bias_a=None, bias_x=None, z=None,
                       seq_start=None, dh_last=None, want_dh0=False, workspace=None, stream=None,
                       out=None):
    """Gradients of sum(dout * y) [+ sum(dh_last * h_last)] for
    ssm_gated_scan_fwd with the same inputs, from the ``chunk_states`` it
    filled.  Returns a dict: du, dgate_a, dgate_x, dz (activation dtype; dz
    only with z); dA, dbias_a, dbias_x (d_in,) fp32 (the biases' only with
    them); dh0 (b, d_in) fp32 when want_dh0.  ``out``: a dict of tensors to
    write into, by those names."""
    dev = _device_of(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be (b, L, d_in)")
    shape, act, f32 = u.shape, u.dtype, torch.float32
    b, L, d = shape
    code = _dtype_code(u)
    ins = _gated_inputs(u, gate_a, gate_x, A, bias_a, bias_x, z, shape, dev)
    _need(seq_start, "seq_start", (b, L), torch.uint8, dev)
    _need(dh_last, "dh_last", (b, d), f32, dev)
    if states is None:
        raise TypeError("states: expected the chunk_states of ssm_gated_scan_fwd")
    states = _chunk_states(states, "states", b, L, d, dev)
    pool = _Pool(dev, stream)
    if A is None:
        raise TypeError("A: expected a torch.Tensor")
    likes = dict(du=u, dgate_a=u, dgate_x=u)
    if z is not None:
        likes["dz"] = u
    params = dict(dA=A)
    if bias_a is not None:
        params["dbias_a"] = bias_a
    if bias_x is not None:
        params["dbias_x"] = bias_x
    g = _outputs(out, likes, params, pool, dev)
    if want_dh0:
        dh0 = None if out is None else out.get("dh0")
        _need(dh0, "dh0", (b, d), f32, dev)
        g["dh0"] = pool.new(A, (b, d), f32) if dh0 is None else dh0
    ws, ws_ptr, ws_bytes = _workspace(
        workspace, lambda: _lib.ssm_gated_scan_bwd_workspace_bytes(b, L, d), pool, A)
    grads = [v for k in ("du", "dgate_a", "dgate_x", "dz")
             for v in _rows(g.get(k), k, shape, act, dev)]
    _launch(_lib.ssm_gated_scan_bwd, "ssm_gated_scan_bwd", dev, stream, *ins, _ptr(seq_start),
            *_rows(dout, "dout", shape, act, dev), _ptr(dh_last), *grads, _ptr(g["dA"]),
            _ptr(g.get("dbias_a")), _ptr(g.get("dbias_x")), _ptr(g.get("dh0")), b, L, d, code,
            *states, ws_ptr, ws_bytes)
    return g


def ssm_gated_state_update(state, u, gate_a, gate_x, A, bias_a=None, bias_x=None, z=None, y=None,
                           stream=None):
    """One token of the gated recurrence; state (b, d_in) fp32 is updated in
    place.  u, gate_a, gate_x, z: (b, d_in).  Returns y (b, d_in)."""
    dev = _device_of(u, "u")
    if u.dim() != 2:
        raise ValueError("u must be (b, d_in)")
    shape = u.shape
    code = _dtype_code(u)
    ins = _gated_inputs(u, gate_a, gate_x, A, bias_a, bias_x, z, shape, dev)
    if state is None:
        raise TypeError("state: expected a torch.Tensor")
    _need(state, "state", shape, torch.float32, dev)
    if y is None:
        y = _Pool(dev, stream).like(u)
    _launch(_lib.ssm_gated_state_update, "ssm_gated_state_update", dev, stream, _ptr(state), *ins,
            *_rows(y, "y", shape, u.dtype, dev), shape[0], shape[1], code)
    return y


def _conv_inputs(x, weight, bias, shape, dev):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be (d_in, d_conv)")
    d, K = shape[-1], weight.shape[1]
    _need(weight, "weight", (d, K), torch.float32, dev)
    _need(bias, "bias", (d,), torch.float32, dev)
    return _rows(x, "x", shape, x.dtype, dev), K


def ssm_conv1d_fwd(x, weight, bias=None, silu=True, conv_state=None, conv_state_out=None,
                   seq_start=None, y=None, stream=None):
    """Causal depthwise convolution over a sequence (see include/ssmscan.h).
    x: (b, L, d_in); weight: (d_in, d_conv) fp32; bias: (d_in,) fp32;
    conv_state (the window in front of the first step), conv_state_out (the
    one behind the last; may be conv_state): (b, d_in, d_conv) in x's dtype;
    seq_start: (b, L) uint8.  Returns y (b, L, d_in)."""
    dev = _device_of(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be (b, L, d_in)")
    shape = x.shape
    b, L, d = shape
    code = _dtype_code(x)
    xr, K = _conv_inputs(x, weight, bias, shape, dev)
    _need(conv_state, "conv_state", (b, d, K), x.dtype, dev)
    _need(conv_state_out, "conv_state_out", (b, d, K), x.dtype, dev)
    _need(seq_start, "seq_start", (b, L), torch.uint8, dev)
    if y is None:
        y = _Pool(dev, stream).like(x)
    _launch(_lib.ssm_conv1d_fwd, "ssm_conv1d_fwd", dev, stream, *xr, _ptr(weight), _ptr(bias),
            int(bool(silu)), _ptr(conv_state), _ptr(conv_state_out), _ptr(seq_start),
            *_rows(y, "y", shape, x.dtype, dev), b, L, d, K, code)
    return y


def ssm_conv1d_bwd_workspace_bytes(b: int, L: int, d_in: int, d_conv: int) -> int:
    return int(_lib.ssm_conv1d_bwd_workspace_bytes(b, L, d_in, d_conv))


def ssm_conv1d_bwd(x, weight, dy, bias=None, silu=True, conv_state=None, seq_start=None,
                   workspace=None, stream=None, out=None):
    """Gradients of sum(dy * y) for ssm_conv1d_fwd with the same inputs:
    a dict of dx (b, L, d_in), dweight (d_in, d_conv) fp32 and, with a bias,
    dbias (d_in,) fp32.  ``out``: a dict of tensors to write into."""
    dev = _device_of(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be (b, L, d_in)")
    shape, act, f32 = x.shape, x.dtype, torch.float32
    b, L, d = shape
    code = _dtype_code(x)
    xr, K = _conv_inputs(x, weight, bias, shape, dev)
    _need(conv_state, "conv_state", (b, d, K), act, dev)
    _need(seq_start, "seq_start", (b, L), torch.uint8, dev)
    pool = _Pool(dev, stream)
    params = dict(dweight=weight)
    if bias is not None:
        params["dbias"] = bias
    g = _outputs(out, dict(dx=x), params, pool, dev)
    ws, ws_ptr, ws_bytes = _workspace(
        workspace, lambda: _lib.ssm_conv1d_bwd_workspace_bytes(b, L, d, K), pool, weight)
    _launch(_lib.ssm_conv1d_bwd, "ssm_conv1d_bwd", dev, stream, *xr, _ptr(weight), _ptr(bias),
            int(bool(silu)), _ptr(conv_state), _ptr(seq_start), *_rows(dy, "dy", shape, act, dev),
            *_rows(g["dx"], "dx", shape, act, dev), _ptr(g["dweight"]), _ptr(g.get("dbias")), b, L, d,
            K, code, ws_ptr, ws_bytes)
    return g


def ssm_conv1d_update(conv_state, x, weight, bias=None, silu=True, y=None, stream=None):
    """One token of the convolution; conv_state (b, d_in, d_conv) in x's dtype
    is rolled and x (b, d_in) put last, in place.  Returns y (b, d_in)."""
    dev = _device_of(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be (b, d_in)")
    shape = x.shape
    code = _dtype_code(x)
    xr, K = _conv_inputs(x, weight, bias, shape, dev)
    if conv_state is None:
        raise TypeError("conv_state: expected a torch.Tensor")
    _need(conv_state, "conv_state", (*shape, K), x.dtype, dev)
    if y is None:
        y = _Pool(dev, stream).like(x)
    _launch(_lib.ssm_conv1d_update, "ssm_conv1d_update", dev, stream, _ptr(conv_state), *xr,
            _ptr(weight), _ptr(bias), int(bool(silu)), *_rows(y, "y", shape, x.dtype, dev), shape[0],
            shape[1], K, code)
    return y


def _row_count(shape):
    n = 1
    for s in shape[:-1]:
        n *= s
    return n


def ssm_gated_norm_fwd(x, z, weight, groups=1, eps=1e-5, norm_before_gate=False, y=None, stream=None):
    """RMS norm over `groups` groups of channels with the SiLU gate z (None:
    no gate): rms(x silu(z)) weight, or rms(x) weight silu(z) with
    norm_before_gate.  x, z: (..., d); weight: (d,) fp32.  Returns y like x."""
    dev = _device_of(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be (..., d)")
    shape, act = x.shape, x.dtype
    d = shape[-1]
    code = _dtype_code(x)
    xr, zr = _rows(x, "x", shape, act, dev), _rows(z, "z", shape, act, dev)
    _need(weight, "weight", (d,), torch.float32, dev)
    if y is None:
        y = _Pool(dev, stream).like(x)
    _launch(_lib.ssm_gated_norm_fwd, "ssm_gated_norm_fwd", dev, stream, *xr, *zr, _ptr(weight), groups,
            eps, int(bool(norm_before_gate)), *_rows(y, "y", shape, act, dev), _row_count(shape), d,
            code)
    return y


def ssm_gated_norm_bwd_workspace_bytes(rows: int, d: int, groups: int = 1) -> int:
    return int(_lib.ssm_gated_norm_bwd_workspace_bytes(rows, d, groups))


def ssm_gated_norm_bwd(x, z, weight, dy, groups=1, eps=1e-5, norm_before_gate=False, workspace=None,
                       stream=None, out=None):
    """Gradients of sum(dy * y) for ssm_gated_norm_fwd with the same inputs: a
    dict of dx, dz (with z) like x, and dweight (d,) fp32.  ``out``: a dict of
    tensors to write into."""
    dev = _device_of(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be (..., d)")
    shape, act = x.shape, x.dtype
    d, rows = shape[-1], _row_count(shape)
    code = _dtype_code(x)
    xr, zr = _rows(x, "x", shape, act, dev), _rows(z, "z", shape, act, dev)
    _need(weight, "weight", (d,), torch.float32, dev)
    dyr = _rows(dy, "dy", shape, act, dev)
    pool = _Pool(dev, stream)
    if weight is None:
        raise TypeError("weight: expected a torch.Tensor")
    likes = dict(dx=x) if z is None else dict(dx=x, dz=x)
    g = _outputs(out, likes, dict(dweight=weight), pool, dev)
    ws, ws_ptr, ws_bytes = _workspace(
        workspace, lambda: _lib.ssm_gated_norm_bwd_workspace_bytes(rows, d, groups), pool, weight)
    _launch(_lib.ssm_gated_norm_bwd, "ssm_gated_norm_bwd", dev, stream, *xr, *zr, _ptr(weight), groups,
            eps, int(bool(norm_before_gate)), *dyr, *_rows(g["dx"], "dx", shape, act, dev),
            *_rows(g.get("dz"), "dz", shape, act, dev), _ptr(g["dweight"]), rows, d, code, ws_ptr,
            ws_bytes)
    return g


def ssm_add_norm_fwd(x, residual, weight, scale=None, post_weight=None, eps=1e-5,
                     residual_dtype=None, y=None, residual_out=None, stream=None):
    """residual_out = residual + scale * (post_weight ? rms(x) * post_weight : x)
    and y = rms(residual_out) * weight.  x: (..., d); residual the same in
    fp32 or x's dtype, or None (0); weight, scale, post_weight: (d,) fp32.
    residual_dtype: of residual_out without a residual (default x's).
    Returns (y, residual_out); residual_out may be residual."""
    dev = _device_of(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be (..., d)")
    shape, act, f32 = x.shape, x.dtype, torch.float32
    d = shape[-1]
    code = _dtype_code(x)
    if residual is not None:
        if not isinstance(residual, torch.Tensor):
            raise TypeError("residual: expected a torch.Tensor")
        if residual_dtype is not None and residual_dtype != residual.dtype:
            raise TypeError(f"residual: dtype {residual.dtype}, expected {residual_dtype}")
        residual_dtype = residual.dtype
    elif residual_dtype is None:
        residual_dtype = act if residual_out is None else residual_out.dtype
    if residual_dtype != f32 and residual_dtype != act:
        raise TypeError(f"residual dtype {residual_dtype}: expected fp32 or {act}")
    rcode = SSM_F32 if residual_dtype == f32 else SSM_BF16
    xr = _rows(x, "x", shape, act, dev)
    rr = _rows(residual, "residual", shape, residual_dtype, dev)
    _need(weight, "weight", (d,), f32, dev)
    _need(scale, "scale", (d,), f32, dev)
    _need(post_weight, "post_weight", (d,), f32, dev)
    pool = _Pool(dev, stream)
    if y is None:
        y = pool.like(x)
    if residual_out is None:
        residual_out = pool.like(x, residual_dtype)
    _launch(_lib.ssm_add_norm_fwd, "ssm_add_norm_fwd", dev, stream, *xr, *rr, _ptr(weight),
            _ptr(post_weight), _ptr(scale), eps, *_rows(y, "y", shape, act, dev),
            *_rows(residual_out, "residual_out", shape, residual_dtype, dev), _row_count(shape), d,
            code, rcode)
    return y, residual_out


def ssm_add_norm_bwd_workspace_bytes(rows: int, d: int) -> int:
    return int(_lib.ssm_add_norm_bwd_workspace_bytes(rows, d))


def ssm_add_norm_bwd(x, residual_out, weight, dy, dresidual_out=None, scale=None, post_weight=None,
                     eps=1e-5, want_dresidual=True, workspace=None, stream=None, out=None):
    """Gradients of sum(dy * y) [+ sum(dresidual_out * residual_out)] for
    ssm_add_norm_fwd, from the residual_out it wrote: a dict of dx, dresidual
    (in residual_out's dtype, unless not wanted), dweight and, where given,
    dscale, dpost_weight (d,) fp32.  x may be None without scale and
    post_weight.  ``out``: a dict of tensors to write into; its dresidual may
    be dresidual_out."""
    dev = _device_of(dy, "dy")
    if dy.dim() < 1:
        raise ValueError("dy must be (..., d)")
    shape, act, f32 = dy.shape, dy.dtype, torch.float32
    d, rows = shape[-1], _row_count(shape)
    code = _dtype_code(dy)
    if not isinstance(residual_out, torch.Tensor):
        raise TypeError("residual_out: expected a torch.Tensor")
    res = residual_out.dtype
    if res != f32 and res != act:
        raise TypeError(f"residual dtype {res}: expected fp32 or {act}")
    if x is None and (scale is not None or post_weight is not None):
        raise TypeError("x: expected a torch.Tensor with scale or post_weight")
    xr = _rows(x, "x", shape, act, dev)
    rr = _rows(residual_out, "residual_out", shape, res, dev)
    _need(weight, "weight", (d,), f32, dev)
    _need(scale, "scale", (d,), f32, dev)
    _need(post_weight, "post_weight", (d,), f32, dev)
    dyr = _rows(dy, "dy", shape, act, dev)
    dror = _rows(dresidual_out, "dresidual_out", shape, res, dev)
    pool = _Pool(dev, stream)
    if weight is None:
        raise TypeError("weight: expected a torch.Tensor")
    likes = dict(dx=dy)
    if want_dresidual:
        likes["dresidual"] = residual_out
    params = dict(dweight=weight)
    if post_weight is not None:
        params["dpost_weight"] = post_weight
    if scale is not None:
        params["dscale"] = scale
    g = _outputs(out, likes, params, pool, dev)
    ws, ws_ptr, ws_bytes = _workspace(
        workspace, lambda: _lib.ssm_add_norm_bwd_workspace_bytes(rows, d), pool, weight)
    _launch(_lib.ssm_add_norm_bwd, "ssm_add_norm_bwd", dev, stream, *xr, *rr, _ptr(weight),
            _ptr(post_weight), _ptr(scale), eps, *dyr, *dror, *_rows(g["dx"], "dx", shape, act, dev),
            *_rows(g.get("dresidual"), "dresidual", shape, res, dev), _ptr(g["dweight"]),
            _ptr(g.get("dpost_weight")), _ptr(g.get("dscale")), rows, d, code,
            SSM_F32 if res == f32 else SSM_BF16, ws_ptr, ws_bytes)
    return g


def check_device_errors(stream=None) -> None:
    """Synchronise and raise if a kernel reported a device-side error."""
    _check(_lib.ssm_check_device_errors(_stream(stream)), "ssm_check_device_errors")


def debug_bounds_enabled() -> bool:
    """True when the loaded library is the debug-bounds build."""
    return bool(_lib.ssm_debug_bounds_enabled())


def debug_bounds_self_test(stream=None) -> int:
    """Enqueue the debug-bounds build's self-test (one index one past its
    range: recorded, access skipped); returns the status of the call."""
    return int(_lib.ssm_debug_bounds_self_test(_stream(stream)))
