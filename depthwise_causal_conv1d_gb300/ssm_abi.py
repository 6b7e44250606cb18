"""Raw binding of the state-space operators of ``include/ccu_ssm.h``: the argument structs and
the ``ccu_*`` functions on them (device pointers as ints), and the names of the scan's routes. Needs no PyTorch."""

from __future__ import annotations

import ctypes

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

SCAN_ROUTES = {"auto": 0, "recurrent": 1, "chunked": 2}


class Conv1dPackedArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("ld_x", _i64), ("weight", _vp), ("bias", _vp), ("conv_state", _vp),
                ("stride_s", _i64), ("stride_d", _i64), ("stride_l", _i64), ("cu_seqlens", _vp),
                ("indices", _vp), ("has_initial", _vp), ("out", _vp), ("ld_out", _i64), ("status_dev", _vp),
                ("T", _i64), ("B", _i64), ("D", _i64), ("S", _i64), ("L", _i64), ("W", _i64),
                ("act", _i32), ("reserved", _i32)]


class SelectiveScanArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_stride_t", _i64), ("x_stride_h", _i64), ("dt", _vp), ("dt_stride_t", _i64),
                ("b", _vp), ("b_stride_t", _i64), ("b_stride_g", _i64), ("c", _vp), ("c_stride_t", _i64),
                ("c_stride_g", _i64), ("z", _vp), ("z_stride_t", _i64), ("z_stride_h", _i64), ("A", _vp),
                ("D", _vp), ("dt_bias", _vp), ("cu_seqlens", _vp), ("indices", _vp), ("has_initial", _vp),
                ("state", _vp), ("state_stride_s", _i64), ("out", _vp), ("out_stride_t", _i64),
                ("out_stride_h", _i64), ("workspace", _vp), ("workspace_bytes", _i64), ("status_dev", _vp),
                ("T", _i64), ("n_seq", _i64), ("H", _i64), ("P", _i64), ("K", _i64), ("G", _i64), ("S", _i64),
                ("dt_softplus", _i32), ("route", _i32)]


class SelectiveStateUpdateArgs(ctypes.Structure):
    _fields_ = [("xbc", _vp), ("ld_xbc", _i64), ("conv_weight", _vp), ("conv_bias", _vp), ("conv_state", _vp),
                ("conv_stride_s", _i64), ("conv_stride_d", _i64), ("conv_stride_l", _i64), ("dt", _vp),
                ("dt_stride_n", _i64), ("z", _vp), ("z_stride_n", _i64), ("z_stride_h", _i64), ("A", _vp),
                ("D", _vp), ("dt_bias", _vp), ("indices", _vp), ("state", _vp), ("state_stride_s", _i64),
                ("out", _vp), ("out_stride_n", _i64), ("out_stride_h", _i64), ("workspace", _vp),
                ("workspace_bytes", _i64), ("status_dev", _vp), ("N", _i64), ("H", _i64), ("P", _i64), ("K", _i64), ("G", _i64), ("S", _i64), ("L", _i64), ("W", _i64), ("act", _i32),
                ("dt_softplus", _i32)]


class W4MatmulArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("ld_x", _i64), ("qweight", _vp), ("scales", _vp), ("zeros", _vp), ("out", _vp),
                ("ld_out", _i64), ("M", _i64), ("I", _i64), ("O", _i64), ("group", _i64)]


def declare(lib) -> None:
    """Argument and result types of the entry points on a loaded library."""
    for name, args in (("ccu_causal_conv1d_packed", Conv1dPackedArgs), ("ccu_selective_scan", SelectiveScanArgs),
                       ("ccu_selective_state_update", SelectiveStateUpdateArgs), ("ccu_w4_matmul", W4MatmulArgs)):
        f = getattr(lib, name)
        f.argtypes = [ctypes.POINTER(args), _vp]
        f.restype = ctypes.c_int
    lib.ccu_selective_scan_workspace_bytes.argtypes = [ctypes.POINTER(SelectiveScanArgs)]
    lib.ccu_selective_scan_workspace_bytes.restype = _i64
    lib.ccu_selective_state_update_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64, _i32]
    lib.ccu_selective_state_update_workspace_bytes.restype = _i64
    lib.ccu_selective_scan_select_route.argtypes = [ctypes.POINTER(SelectiveScanArgs)]
    lib.ccu_selective_scan_select_route.restype = _i32


from . import lib  # noqa: E402  (the package loads the library first)

declare(lib)


# ------------------------------------------------------------------ raw C entry points

def ccu_causal_conv1d_packed(args: Conv1dPackedArgs, stream) -> int:
    return lib.ccu_causal_conv1d_packed(ctypes.byref(args), stream)


def ccu_selective_scan(args: SelectiveScanArgs, stream) -> int:
    return lib.ccu_selective_scan(ctypes.byref(args), stream)


def ccu_selective_scan_workspace_bytes(args: SelectiveScanArgs) -> int:
    return lib.ccu_selective_scan_workspace_bytes(ctypes.byref(args))


def ccu_selective_scan_select_route(args: SelectiveScanArgs) -> int:
    return lib.ccu_selective_scan_select_route(ctypes.byref(args))


def ccu_selective_state_update(args: SelectiveStateUpdateArgs, stream) -> int:
    return lib.ccu_selective_state_update(ctypes.byref(args), stream)


def ccu_selective_state_update_workspace_bytes(N, H, P, K, G, has_conv) -> int:
    return lib.ccu_selective_state_update_workspace_bytes(N, H, P, K, G, has_conv)


def ccu_w4_matmul(args: W4MatmulArgs, stream) -> int:
    return lib.ccu_w4_matmul(ctypes.byref(args), stream)
