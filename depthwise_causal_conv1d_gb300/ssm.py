"""Binding of the state-space operators of ``include/ccu_ssm.h``.

Argument marshalling only, as in the package's ``__init__``: the raw ``ccu_*`` functions
take the C structs below (device pointers as ints), the torch-level functions check tensors,
fill a struct and launch on the current stream of the tensors' device. Scratch memory comes
from torch's allocator unless the caller passes a ``workspace``.
"""

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
                ("workspace_bytes", _i64), ("status_dev", _vp), ("N", _i64), ("H", _i64), ("P", _i64),
                ("K", _i64), ("G", _i64), ("S", _i64), ("L", _i64), ("W", _i64), ("act", _i32),
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
    lib.ccu_selective_scan_select_route.argtypes = [ctypes.POINTER(SelectiveScanArgs)]
    lib.ccu_selective_scan_select_route.restype = _i32
    lib.ccu_selective_state_update_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64, _i32]
    lib.ccu_selective_state_update_workspace_bytes.restype = _i64


from . import _ACTIVATIONS, lib, raise_for_status  # noqa: E402  (the package loads the library first)

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


# ------------------------------------------------------------------ torch-level ops

def _check(torch, dev, name, t, dtype, shape, contiguous=False):
    """One tensor of a call: its type, its place, and its shape (None matches any size)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor" if not t.is_cuda else
                         f"{name} is on {t.device}: all tensors of a call must be on one device")
    if t.requires_grad:
        raise ValueError(f"{name} requires grad: the operator is inference-only (autograd unsupported)")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must be [{', '.join('*' if w is None else str(w) for w in shape)}], "
                         f"got {list(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _unit_last(name, t):
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")


def _launch(torch, dev, entry, args):
    """Runs a C entry point on the current stream of device ``dev`` (its launches go to the
    current device)."""
    if dev == torch.cuda.current_device():
        st = entry(ctypes.byref(args), torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = entry(ctypes.byref(args), torch.cuda.current_stream(dev).cuda_stream)
    if st:
        raise_for_status(st)


def _activation(activation):
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of None, 'identity', 'silu', 'swish'; got {activation!r}")
    return _ACTIVATIONS[activation]


def causal_conv1d_packed(x, weight, bias=None, activation=None, *, cu_seqlens, conv_state=None,
                         conv_state_indices=None, has_initial_state=None, out=None, status=None):
    """Causal depthwise convolution of packed prompts: ``x`` BF16 ``[T, D]`` (any row stride)
    holds the sequences ``cu_seqlens[b]..cu_seqlens[b+1]`` (int32 ``[B + 1]`` on the device).

    With a ``conv_state`` (BF16 ``[S, D, L]``) sequence ``b`` continues from the entries in its
    slot (``conv_state_indices[b]``, or ``b``) when ``has_initial_state[b]`` (int32 ``[B]``) is
    nonzero, and leaves its last L inputs there, ready for ``causal_conv1d_update`` or
    ``selective_state_update``. A slot of -1 is a padding sequence: outputs +0, no state touched.
    Returns BF16 ``[T, D]``; rows outside every sequence are left unwritten.
    """
    import torch

    act = _activation(activation)
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev, bf16, i32 = x.get_device(), torch.bfloat16, torch.int32
    xp = _check(torch, dev, "x", x, bf16, (None, None))
    _unit_last("x", x)
    T, D = x.shape
    wp = _check(torch, dev, "weight", weight, bf16, (D, None), True)
    W = weight.shape[1]
    bp = None if bias is None else _check(torch, dev, "bias", bias, bf16, (D,), True)
    cp = _check(torch, dev, "cu_seqlens", cu_seqlens, i32, (None,), True)
    B = cu_seqlens.shape[0] - 1
    if B < 0:
        raise ValueError("cu_seqlens must have at least one entry")
    sp, S, L, strides = None, 0, 0, (0, 0, 0)
    if conv_state is not None:
        sp = _check(torch, dev, "conv_state", conv_state, bf16, (None, D, None))
        S, _, L = conv_state.shape
        strides = conv_state.stride()
    ip = None if conv_state_indices is None else _check(torch, dev, "conv_state_indices", conv_state_indices, i32, (B,), True)
    hp = None if has_initial_state is None else _check(torch, dev, "has_initial_state", has_initial_state, i32, (B,), True)
    tp = None if status is None else _check(torch, dev, "status", status, i32, (1,))
    if out is None:
        out = torch.empty((T, D), dtype=bf16, device=x.device)
    op = _check(torch, dev, "out", out, bf16, (T, D))
    _unit_last("out", out)
    args = Conv1dPackedArgs(xp, x.stride(0), wp, bp, sp, *strides, cp, ip, hp, op, out.stride(0), tp,
                            T, B, D, S, L, W, act, 0)
    _launch(torch, dev, lib.ccu_causal_conv1d_packed, args)
    return out


def selective_scan(x, dt, A, B, C, *, cu_seqlens, ssm_state, D=None, z=None, dt_bias=None, dt_softplus=True,
                   state_indices=None, has_initial_state=None, out=None, workspace=None, status=None,
                   route: str = "auto"):
    """Selective state space scan of packed prompts.

    ``x`` BF16 ``[T, H, P]``, ``dt`` BF16 ``[T, H]``, ``B`` and ``C`` BF16 ``[T, G, K]`` and the gate
    ``z`` (BF16 ``[T, H, P]`` or None) may be slices of wider rows (unit stride along the last
    dimension); ``A``, ``D``, ``dt_bias`` FP32 ``[H]``. Per head the state ``s[P, K]`` runs as
    ``s = exp(d A) s + d x B``, ``y = C s + D x`` with ``d = softplus(dt + dt_bias)`` (``dt + dt_bias``
    without ``dt_softplus``), gated by ``z * sigmoid(z)``. Sequences, slots and initial states are as in
    ``causal_conv1d_packed``; ``ssm_state`` is FP32 ``[S, H, P, K]`` (slots may be further apart) and
    receives the state after each sequence. Returns BF16 ``[T, H, P]``.

    ``workspace`` (uint8, at least ``ccu_selective_scan_workspace_bytes``) replaces the scratch
    the call otherwise takes from torch; ``route`` forces a kernel ("recurrent", "chunked").
    """
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if route not in SCAN_ROUTES:
        raise ValueError(f"route must be one of {sorted(SCAN_ROUTES)}")
    dev, bf16, f32, i32 = x.get_device(), torch.bfloat16, torch.float32, torch.int32
    xp = _check(torch, dev, "x", x, bf16, (None, None, None))
    T, H, P = x.shape
    dp = _check(torch, dev, "dt", dt, bf16, (T, H))
    bp = _check(torch, dev, "B", B, bf16, (T, None, None))
    _, G, K = B.shape
    cp = _check(torch, dev, "C", C, bf16, (T, G, K))
    for name, t in (("x", x), ("dt", dt), ("B", B), ("C", C)):
        _unit_last(name, t)
    zp, zs = None, (0, 0)
    if z is not None:
        zp, zs = _check(torch, dev, "z", z, bf16, (T, H, P)), z.stride()
        _unit_last("z", z)
    ap = _check(torch, dev, "A", A, f32, (H,), True)
    Dp = None if D is None else _check(torch, dev, "D", D, f32, (H,), True)
    tb = None if dt_bias is None else _check(torch, dev, "dt_bias", dt_bias, f32, (H,), True)
    up = _check(torch, dev, "cu_seqlens", cu_seqlens, i32, (None,), True)
    n_seq = cu_seqlens.shape[0] - 1
    if n_seq < 0:
        raise ValueError("cu_seqlens must have at least one entry")
    sp = _check(torch, dev, "ssm_state", ssm_state, f32, (None, H, P, K))
    S = ssm_state.shape[0]
    if S > 0 and not ssm_state[0].is_contiguous():
        raise ValueError("a slot of ssm_state must be contiguous")
    ip = None if state_indices is None else _check(torch, dev, "state_indices", state_indices, i32, (n_seq,), True)
    hp = None if has_initial_state is None else _check(torch, dev, "has_initial_state", has_initial_state, i32, (n_seq,), True)
    tp = None if status is None else _check(torch, dev, "status", status, i32, (1,))
    if out is None:
        out = torch.empty((T, H, P), dtype=bf16, device=x.device)
    op = _check(torch, dev, "out", out, bf16, (T, H, P))
    _unit_last("out", out)
    xs, os = x.stride(), out.stride()
    args = SelectiveScanArgs(xp, xs[0], xs[1], dp, dt.stride(0), bp, B.stride(0), B.stride(1), cp, C.stride(0),
                             C.stride(1), zp, zs[0], zs[1], ap, Dp, tb, up, ip, hp, sp, ssm_state.stride(0), op,
                             os[0], os[1], None, 0, tp, T, n_seq, H, P, K, G, S, 1 if dt_softplus else 0,
                             SCAN_ROUTES[route])
    if workspace is None:
        with torch.cuda.device(dev):
            need = lib.ccu_selective_scan_workspace_bytes(ctypes.byref(args))
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if workspace is not None:
        args.workspace = _check(torch, dev, "workspace", workspace, torch.uint8, (None,), True)
        args.workspace_bytes = workspace.shape[0]
    _launch(torch, dev, lib.ccu_selective_scan, args)
    return out


def selective_state_update(xbc, dt, A, ssm_state, conv_state=None, conv_weight=None, conv_bias=None, activation=None, *,
                           D=None, z=None, dt_bias=None, dt_softplus=True, groups=1, state_indices=None, out=None,
                           workspace=None, status=None):
    """One token per row: convolution step and state step, both in place on the row's slot.

    ``xbc`` BF16 ``[N, H*P + 2*G*K]`` (any row stride) holds x, then B, then C of the ``groups`` G.
    With ``conv_weight`` (BF16 ``[H*P + 2*G*K, W]``) it goes through the step of
    ``causal_conv1d_update`` on ``conv_state`` (BF16 ``[S, H*P + 2*G*K, L]``) first, its result kept in
    32 bits; without, it is taken as is. Then one step of ``selective_scan`` on ``ssm_state``
    (FP32 ``[S, H, P, K]``). Returns BF16 ``[N, H, P]``. ``state_indices`` (int32 ``[N]``) picks the
    slots, -1 marking padding rows (output +0).
    """
    import torch

    if not isinstance(xbc, torch.Tensor):
        raise TypeError("xbc must be a torch.Tensor")
    dev, bf16, f32, i32 = xbc.get_device(), torch.bfloat16, torch.float32, torch.int32
    sp = _check(torch, dev, "ssm_state", ssm_state, f32, (None, None, None, None))
    S, H, P, K = ssm_state.shape
    if S > 0 and not ssm_state[0].is_contiguous():
        raise ValueError("a slot of ssm_state must be contiguous")
    G = groups
    channels = H * P + 2 * G * K
    xp = _check(torch, dev, "xbc", xbc, bf16, (None, channels))
    _unit_last("xbc", xbc)
    N = xbc.shape[0]
    wp = kp = cp = None
    act, L, W, cs = 0, 0, 0, (0, 0, 0)
    if conv_weight is not None:
        act = _activation(activation)
        wp = _check(torch, dev, "conv_weight", conv_weight, bf16, (channels, None), True)
        W = conv_weight.shape[1]
        if conv_state is None:
            raise ValueError("conv_weight needs a conv_state")
        cp = _check(torch, dev, "conv_state", conv_state, bf16, (S, channels, None))
        L, cs = conv_state.shape[2], conv_state.stride()
        kp = None if conv_bias is None else _check(torch, dev, "conv_bias", conv_bias, bf16, (channels,), True)
    elif conv_state is not None or conv_bias is not None:
        raise ValueError("conv_state and conv_bias need a conv_weight")
    dp = _check(torch, dev, "dt", dt, bf16, (N, H))
    _unit_last("dt", dt)
    zp, zs = None, (0, 0)
    if z is not None:
        zp, zs = _check(torch, dev, "z", z, bf16, (N, H, P)), z.stride()
        _unit_last("z", z)
    ap = _check(torch, dev, "A", A, f32, (H,), True)
    Dp = None if D is None else _check(torch, dev, "D", D, f32, (H,), True)
    tb = None if dt_bias is None else _check(torch, dev, "dt_bias", dt_bias, f32, (H,), True)
    ip = None if state_indices is None else _check(torch, dev, "state_indices", state_indices, i32, (N,), True)
    tp = None if status is None else _check(torch, dev, "status", status, i32, (1,))
    if out is None:
        out = torch.empty((N, H, P), dtype=bf16, device=xbc.device)
    op = _check(torch, dev, "out", out, bf16, (N, H, P))
    _unit_last("out", out)
    if workspace is None and wp is not None:
        workspace = torch.empty(4 * N * channels, dtype=torch.uint8, device=xbc.device)
    ws, wn = None, 0
    if workspace is not None:
        ws, wn = _check(torch, dev, "workspace", workspace, torch.uint8, (None,), True), workspace.shape[0]
    os = out.stride()
    args = SelectiveStateUpdateArgs(xp, xbc.stride(0), wp, kp, cp, *cs, dp, dt.stride(0), zp, zs[0], zs[1], ap, Dp, tb,
                                    ip, sp, ssm_state.stride(0), op, os[0], os[1], ws, wn, tp, N, H, P, K, G, S, L, W,
                                    act, 1 if dt_softplus else 0)
    _launch(torch, dev, lib.ccu_selective_state_update, args)
    return out


def w4_matmul(x, qweight, scales, zeros=None, *, out=None):
    """``x @ W.T`` for a matrix of 4-bit weights: ``x`` BF16 ``[M, I]`` (any row stride), ``qweight``
    uint8 ``[O, I // 2]`` (input 2j in the low half of byte j), ``scales`` and ``zeros`` BF16
    ``[O, I // group]`` with groups of 32, 64 or 128 inputs; ``W = (q - zero) * scale``, zero 8 when
    ``zeros`` is None. Returns BF16 ``[M, O]``. See ``w4_quantize``.
    """
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev, bf16 = x.get_device(), torch.bfloat16
    xp = _check(torch, dev, "x", x, bf16, (None, None))
    _unit_last("x", x)
    M, I = x.shape  # noqa: E741
    if I % 2:
        raise ValueError("x must have an even number of columns")
    qp = _check(torch, dev, "qweight", qweight, torch.uint8, (None, I // 2), True)
    O = qweight.shape[0]  # noqa: E741
    sp = _check(torch, dev, "scales", scales, bf16, (O, None), True)
    groups = scales.shape[1]
    if groups < 1 or I % groups:
        raise ValueError(f"scales must split the {I} inputs into equal groups, got {groups}")
    zp = None if zeros is None else _check(torch, dev, "zeros", zeros, bf16, (O, groups), True)
    if out is None:
        out = torch.empty((M, O), dtype=bf16, device=x.device)
    op = _check(torch, dev, "out", out, bf16, (M, O))
    _unit_last("out", out)
    args = W4MatmulArgs(xp, x.stride(0), qp, sp, zp, op, out.stride(0), M, I, O, I // groups)
    _launch(torch, dev, lib.ccu_w4_matmul, args)
    return out


def w4_quantize(weight, group=128, symmetric=True):
    """4-bit form of a weight ``[O, I]`` for ``w4_matmul``: ``(qweight, scales, zeros)``.

    Symmetric: zero 8 (``zeros`` is None), scale ``max|w| / 7`` of the group. Else the group's
    range is spread over 0..15 with an integer zero point. Done once per weight, on the
    weight's device; the scales are rounded to BF16 before the weights are divided by them.
    """
    import torch

    if weight.dim() != 2 or group not in (32, 64, 128) or weight.shape[1] % group:
        raise ValueError("weight must be [O, I] with I a multiple of group (32, 64 or 128)")
    O, I = weight.shape  # noqa: E741
    w = weight.float().view(O, I // group, group)
    if symmetric:
        scale = w.abs().amax(-1) / 7
        zero = torch.full_like(scale, 8.0)
    else:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        scale = (hi - lo) / 15
        zero = None
    scale = torch.where(scale > 0, scale, torch.ones_like(scale)).to(torch.bfloat16)
    if zero is None:
        zero = (-lo / scale.float()).round().clamp(0, 15)
    q = (w / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8).view(O, I)
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return packed, scale, None if symmetric else zero.to(torch.bfloat16)
