"""Torch-level calls of the state-space operators of ``include/ccu_ssm.h``.

Argument marshalling only, as in the package's ``__init__``: the functions check tensors,
fill a struct of ``ssm_abi`` and launch on the current stream of the tensors' device. Scratch memory comes
from torch's allocator unless the caller passes a ``workspace``. The package imports this module (and PyTorch) at the
first use of one of them.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import _ACTIVATIONS, lib, raise_for_status
from .ssm_abi import SCAN_ROUTES, Conv1dPackedArgs, SelectiveScanArgs, SelectiveStateUpdateArgs, W4MatmulArgs

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64

# ------------------------------------------------------------------ torch-level ops
#
# A decode step makes a few of these calls per layer, so their host time counts: a check that
# passes costs a handful of attribute reads, and the struct is packed in one go (_Entry).

class _Entry:
    """A C entry point called with its struct as packed bytes (64-bit members, then 32-bit ones)."""

    def __init__(self, name, args):
        form = struct.Struct("=" + "".join("q" if ctypes.sizeof(t) == 8 else "f" if t is ctypes.c_float else "i" for _, t in args._fields_))
        assert form.size == ctypes.sizeof(args)
        self.pack = form.pack
        self.call = lib[name]  # a function object of its own: it takes bytes
        self.call.argtypes = [ctypes.c_char_p, _vp]
        self.call.restype = ctypes.c_int

    def launch(self, dev, packed):
        """On the current stream of device ``dev`` (the library launches on the current device)."""
        if dev == torch.cuda.current_device():
            st = self.call(packed, _raw_stream(dev))
        else:
            with torch.cuda.device(dev):
                st = self.call(packed, _raw_stream(dev))
        if st:
            raise_for_status(st)


_raw_stream = torch._C._cuda_getCurrentRawStream
_CONV = _Entry("ccu_causal_conv1d_packed", Conv1dPackedArgs)
_SCAN = _Entry("ccu_selective_scan", SelectiveScanArgs)
_STEP = _Entry("ccu_selective_state_update", SelectiveStateUpdateArgs)
_W4 = _Entry("ccu_w4_matmul", W4MatmulArgs)
_scan_workspace = lib["ccu_selective_scan_workspace_bytes"]
_scan_workspace.argtypes = [ctypes.c_char_p]
_scan_workspace.restype = _i64

_bf16, _f32, _i32t, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _sizes(name, t, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(t.shape)}")
    return t.shape


def _check(dev, name, t, dtype, shape, contiguous=False):
    """One tensor of a call: its type, its place and its shape. Returns its address."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and dev >= 0 and t.shape == shape
            and not t.requires_grad and (not contiguous or t.is_contiguous())):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}: all tensors of a call must be on one device")
    if t.requires_grad:
        raise ValueError(f"{name} requires grad: the operator is inference-only (autograd unsupported)")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _maybe(dev, name, t, dtype, shape):
    """An optional contiguous tensor: its address, 0 for None."""
    return 0 if t is None else _check(dev, name, t, dtype, shape, True)


def _strides(name, t):
    """The strides of a tensor with unit stride along its last dimension."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return st


def _slot_stride(state, H, P, K, name="ssm_state"):
    """How far apart the slots of a state are; each slot is contiguous."""
    st = state.stride()
    if st[1:] != (P * K, K, 1) and state.shape[0] > 0 and not state[0].is_contiguous():
        raise ValueError(f"a slot of {name} must be contiguous")
    return st[0]


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
    act = _activation(activation)
    T, D = _sizes("x", x, 2)
    dev = x.get_device()
    xp = _check(dev, "x", x, _bf16, (T, D))
    W = _sizes("weight", weight, 2)[1]
    wp = _check(dev, "weight", weight, _bf16, (D, W), True)
    bp = _maybe(dev, "bias", bias, _bf16, (D,))
    B = _sizes("cu_seqlens", cu_seqlens, 1)[0] - 1
    if B < 0:
        raise ValueError("cu_seqlens must have at least one entry")
    cp = _check(dev, "cu_seqlens", cu_seqlens, _i32t, (B + 1,), True)
    sp, S, L, strides = 0, 0, 0, (0, 0, 0)
    if conv_state is not None:
        S, _, L = _sizes("conv_state", conv_state, 3)
        sp = _check(dev, "conv_state", conv_state, _bf16, (S, D, L))
        strides = conv_state.stride()
    ip = _maybe(dev, "conv_state_indices", conv_state_indices, _i32t, (B,))
    hp = _maybe(dev, "has_initial_state", has_initial_state, _i32t, (B,))
    tp = _maybe(dev, "status", status, _i32t, (1,))
    if out is None:
        out = x.new_empty((T, D))
    op = _check(dev, "out", out, _bf16, (T, D))
    _CONV.launch(dev, _CONV.pack(xp, _strides("x", x)[0], wp, bp, sp, *strides, cp, ip, hp, op, _strides("out", out)[0], tp,
                                 T, B, D, S, L, W, act, 0))
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
    the call otherwise takes from torch; ``route`` forces a kernel ("recurrent", "chunked"). Both compute in
    32 bits; the chunked one, which "auto" takes for prompts where it serves (P and K multiples of 8, K up to 128,
    rows on 16-byte boundaries), gives the factors of the outputs' products 16 bits each, and may give NaN
    where an infinite input makes an infinity.
    """
    if route not in SCAN_ROUTES:
        raise ValueError(f"route must be one of {sorted(SCAN_ROUTES)}")
    T, H, P = _sizes("x", x, 3)
    dev = x.get_device()
    xp = _check(dev, "x", x, _bf16, (T, H, P))
    dp = _check(dev, "dt", dt, _bf16, (T, H))
    _, G, K = _sizes("B", B, 3)
    bp = _check(dev, "B", B, _bf16, (T, G, K))
    cp = _check(dev, "C", C, _bf16, (T, G, K))
    xs, ds, bs, cs = _strides("x", x), _strides("dt", dt), _strides("B", B), _strides("C", C)
    zp, zs = 0, (0, 0)
    if z is not None:
        zp, zs = _check(dev, "z", z, _bf16, (T, H, P)), _strides("z", z)
    ap = _check(dev, "A", A, _f32, (H,), True)
    Dp = _maybe(dev, "D", D, _f32, (H,))
    tb = _maybe(dev, "dt_bias", dt_bias, _f32, (H,))
    n_seq = _sizes("cu_seqlens", cu_seqlens, 1)[0] - 1
    if n_seq < 0:
        raise ValueError("cu_seqlens must have at least one entry")
    up = _check(dev, "cu_seqlens", cu_seqlens, _i32t, (n_seq + 1,), True)
    S = _sizes("ssm_state", ssm_state, 4)[0]
    sp = _check(dev, "ssm_state", ssm_state, _f32, (S, H, P, K))
    ss = _slot_stride(ssm_state, H, P, K)
    ip = _maybe(dev, "state_indices", state_indices, _i32t, (n_seq,))
    hp = _maybe(dev, "has_initial_state", has_initial_state, _i32t, (n_seq,))
    tp = _maybe(dev, "status", status, _i32t, (1,))
    if out is None:
        out = x.new_empty((T, H, P))
    op = _check(dev, "out", out, _bf16, (T, H, P))
    os = _strides("out", out)
    head = (xp, xs[0], xs[1], dp, ds[0], bp, bs[0], bs[1], cp, cs[0], cs[1], zp, zs[0], zs[1], ap, Dp, tb, up, ip, hp, sp,
            ss, op, os[0], os[1])
    tail = (tp, T, n_seq, H, P, K, G, S, 1 if dt_softplus else 0, SCAN_ROUTES[route])
    wp, wn = 0, 0
    if workspace is not None:
        wn = _sizes("workspace", workspace, 1)[0]
        wp = _check(dev, "workspace", workspace, _u8, (wn,), True)
    else:
        with torch.cuda.device(dev):
            wn = _scan_workspace(_SCAN.pack(*head, 0, 0, *tail))
        if wn > 0:
            workspace = x.new_empty((wn + 1) // 2)
            wp = workspace.data_ptr()
        else:
            wn = 0  # none, or a declined call
    _SCAN.launch(dev, _SCAN.pack(*head, wp, wn, *tail))
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
    slots, -1 marking padding rows (output +0). ``workspace`` (uint8, 4 bytes for every entry of
    ``xbc``) replaces the scratch the convolution otherwise takes from torch.
    """
    S, H, P, K = _sizes("ssm_state", ssm_state, 4)
    N = _sizes("xbc", xbc, 2)[0]
    channels = H * P + 2 * groups * K
    dev = xbc.get_device()
    xp = _check(dev, "xbc", xbc, _bf16, (N, channels))
    sp = _check(dev, "ssm_state", ssm_state, _f32, (S, H, P, K))
    wp = kp = cp = act = L = W = ws = wn = 0
    cs = (0, 0, 0)
    if conv_weight is not None:
        act = _activation(activation)
        W = _sizes("conv_weight", conv_weight, 2)[1]
        wp = _check(dev, "conv_weight", conv_weight, _bf16, (channels, W), True)
        if conv_state is None:
            raise ValueError("conv_weight needs a conv_state")
        L = _sizes("conv_state", conv_state, 3)[2]
        cp, cs = _check(dev, "conv_state", conv_state, _bf16, (S, channels, L)), conv_state.stride()
        kp = _maybe(dev, "conv_bias", conv_bias, _bf16, (channels,))
        if workspace is None:
            workspace = xbc.new_empty(2 * N * channels)  # as BF16 entries
            ws, wn = workspace.data_ptr(), 4 * N * channels
        else:
            wn = _sizes("workspace", workspace, 1)[0]
            ws = _check(dev, "workspace", workspace, _u8, (wn,), True)
    elif conv_state is not None or conv_bias is not None:
        raise ValueError("conv_state and conv_bias need a conv_weight")
    dp = _check(dev, "dt", dt, _bf16, (N, H))
    zp, zs = 0, (0, 0)
    if z is not None:
        zp, zs = _check(dev, "z", z, _bf16, (N, H, P)), _strides("z", z)
    ap = _check(dev, "A", A, _f32, (H,), True)
    Dp = _maybe(dev, "D", D, _f32, (H,))
    tb = _maybe(dev, "dt_bias", dt_bias, _f32, (H,))
    ip = _maybe(dev, "state_indices", state_indices, _i32t, (N,))
    tp = _maybe(dev, "status", status, _i32t, (1,))
    if out is None:
        out = xbc.new_empty((N, H, P))
    op = _check(dev, "out", out, _bf16, (N, H, P))
    os = _strides("out", out)
    _STEP.launch(dev, _STEP.pack(xp, _strides("xbc", xbc)[0], wp, kp, cp, *cs, dp, _strides("dt", dt)[0], zp, zs[0], zs[1], ap,
                                 Dp, tb, ip, sp, _slot_stride(ssm_state, H, P, K), op, os[0], os[1], ws, wn, tp, N, H, P, K,
                                 groups, S, L, W, act, 1 if dt_softplus else 0))
    return out


def w4_matmul(x, qweight, scales, zeros=None, *, out=None):
    """``x @ W.T`` for a matrix of 4-bit weights: ``x`` BF16 ``[M, I]`` (any row stride), ``qweight``
    uint8 ``[O, I // 2]`` (input 2j in the low half of byte j), ``scales`` and ``zeros`` BF16
    ``[O, I // group]`` with groups of 32, 64 or 128 inputs; ``W = (q - zero) * scale``, zero 8 when
    ``zeros`` is None. Returns BF16 ``[M, O]``. See ``w4_quantize``.
    """
    M, I = _sizes("x", x, 2)  # noqa: E741
    dev = x.get_device()
    xp = _check(dev, "x", x, _bf16, (M, I))
    O, groups = _sizes("scales", scales, 2)  # noqa: E741
    if I % 2 or groups < 1 or I % groups:
        raise ValueError(f"scales must split the {I} inputs into equal groups, got {groups}")
    qp = _check(dev, "qweight", qweight, _u8, (O, I // 2), True)
    sp = _check(dev, "scales", scales, _bf16, (O, groups), True)
    zp = _maybe(dev, "zeros", zeros, _bf16, (O, groups))
    if out is None:
        out = x.new_empty((M, O))
    op = _check(dev, "out", out, _bf16, (M, O))
    _W4.launch(dev, _W4.pack(xp, _strides("x", x)[0], qp, sp, zp, op, _strides("out", out)[0], M, I, O, I // groups))
    return out


def w4_quantize(weight, group=128, symmetric=True):
    """4-bit form of a weight ``[O, I]`` for ``w4_matmul``: ``(qweight, scales, zeros)``.

    Symmetric: zero 8 (``zeros`` is None), scale ``max|w| / 7`` of the group. Else the group's
    range is spread over 0..15 with an integer zero point. Done once per weight, on the
    weight's device; the scales are rounded to BF16 before the weights are divided by them.
    """
    if weight.dim() != 2 or group not in (32, 64, 128) or weight.shape[1] % group:
        raise ValueError("weight must be [O, I] with I a multiple of group (32, 64 or 128)")
    O, I = weight.shape  # noqa: E741
    w = weight.detach().float().view(O, I // group, group)
    if symmetric:
        scale = w.abs().amax(-1) / 7
        zero = torch.full_like(scale, 8.0)
    else:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        scale = (hi - lo) / 15
        zero = None
    scale = scale.to(torch.bfloat16)
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))  # of zeros, and of what rounds to none
    if zero is None:
        zero = (-lo / scale.float()).round().clamp(0, 15)
    q = (w / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8).view(O, I)
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return packed, scale, None if symmetric else zero.to(torch.bfloat16)
