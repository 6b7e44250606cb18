"""Torch-level calls of the gated delta rule and of the norms around a layer (``include/ccu_ssm.h``).

Argument marshalling only, with the checks and the launch of ``ssm``: on the current stream of the tensors' device, scratch
memory from torch's allocator unless the caller passes a ``workspace``. The package imports this module (and PyTorch) at the
first use of one of them.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import lib
from .ssm import _Entry, _activation, _bf16, _check, _f32, _i32t, _maybe, _sizes, _slot_stride, _strides, _u8
from .ssm_abi import SCAN_ROUTES, GatedDeltaRuleArgs, GatedDeltaUpdateArgs, GatedRmsNormArgs, ResidualRmsNormArgs

_RULE = _Entry("ccu_gated_delta_rule", GatedDeltaRuleArgs)
_STEP = _Entry("ccu_gated_delta_update", GatedDeltaUpdateArgs)
_GATED = _Entry("ccu_gated_rms_norm", GatedRmsNormArgs)
_RESIDUAL = _Entry("ccu_residual_rms_norm", ResidualRmsNormArgs)
_rule_workspace = lib["ccu_gated_delta_rule_workspace_bytes"]
_rule_workspace.argtypes = [ctypes.c_char_p]
_rule_workspace.restype = ctypes.c_int64

_TYPES = {_bf16: 0, _f32: 1}  # ccu_dtype_t


def _single(v):
    """A number in 32 bits, infinite where it overflows: the entry points decline that by name."""
    return ctypes.c_float(v).value


def _scale(scale, K):
    if scale is None:
        return K ** -0.5 if K > 0 else 0.0
    v = _single(scale)
    if not math.isfinite(v) or v == 0:  # 0 would be the entry point's default
        raise ValueError(f"scale must be finite and not 0 in 32 bits, got {scale}")
    return v


def _out(dev, like, out, shape):
    """The output, a new one beside ``like`` unless given, its address and its strides."""
    if out is None:
        out = like.new_empty(shape)
        return out, out.data_ptr(), out.stride()
    return out, _check(dev, "out", out, _bf16, shape), _strides("out", out)


def _type(name, t):
    """ccu_dtype_t of a BF16 or FP32 tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _TYPES:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return _TYPES[t.dtype]


def gated_delta_rule(q, k, v, a, b, A, *, cu_seqlens, state, dt_bias=None, scale=None, qk_norm=True, state_indices=None,
                     has_initial_state=None, out=None, workspace=None, status=None, route: str = "auto"):
    """Gated delta rule of packed prompts.

    ``q`` and ``k`` BF16 ``[T, G, K]``, ``v`` BF16 ``[T, H, P]``, ``a`` and ``b`` BF16 ``[T, H]`` may be slices of wider
    rows (unit stride along the last dimension); head h takes the q and k of group ``h // (H / G)``. ``A`` and
    ``dt_bias`` FP32 ``[H]``. Per head the state ``s[P, K]`` runs as ``s = exp(A softplus(a + dt_bias)) s``,
    ``u = sigmoid(b) (v - s k)``, ``s = s + u k^T``, ``out = scale s q``, with q and k brought to unit length
    (``qk_norm``; 1e-6 is added to the sum of squares) and ``scale`` 1 / sqrt(K) unless given. Sequences, slots and initial states are as in
    ``causal_conv1d_packed``; ``state`` is FP32 ``[S, H, P, K]`` (slots may be further apart) and receives the state
    after each sequence. Returns BF16 ``[T, H, P]``; rows outside every sequence are left unwritten.

    ``workspace`` (uint8, at least ``ccu_gated_delta_rule_workspace_bytes``) replaces the scratch the call otherwise
    takes from torch (long sequences of few heads need some, and those that leave many SMs idle); ``route`` forces a kernel ("recurrent", "chunked"). Both hold the state and what goes into
    it, and the sums of the outputs, in 32 bits; the chunked one, which "auto" takes for prompts where it serves (P and K multiples of 8, K up to 128,
    rows and slots on 16-byte boundaries), gives NaN from its token on where an input or a key's square is infinite.
    """
    if route not in SCAN_ROUTES:
        raise ValueError(f"route must be one of {sorted(SCAN_ROUTES)}")
    T, H, P = _sizes("v", v, 3)
    dev = v.get_device()
    vp = _check(dev, "v", v, _bf16, (T, H, P))
    _, G, K = _sizes("k", k, 3)
    kp = _check(dev, "k", k, _bf16, (T, G, K))
    qp = _check(dev, "q", q, _bf16, (T, G, K))
    ap = _check(dev, "a", a, _bf16, (T, H))
    bp = _check(dev, "b", b, _bf16, (T, H))
    qs, ks, vs, as_, bs = _strides("q", q), _strides("k", k), _strides("v", v), _strides("a", a), _strides("b", b)
    Ap = _check(dev, "A", A, _f32, (H,), True)
    tb = _maybe(dev, "dt_bias", dt_bias, _f32, (H,))
    n_seq = _sizes("cu_seqlens", cu_seqlens, 1)[0] - 1
    if n_seq < 0:
        raise ValueError("cu_seqlens must have at least one entry")
    up = _check(dev, "cu_seqlens", cu_seqlens, _i32t, (n_seq + 1,), True)
    S = _sizes("state", state, 4)[0]
    sp = _check(dev, "state", state, _f32, (S, H, P, K))
    ss = _slot_stride(state, H, P, K, "state")
    ip = _maybe(dev, "state_indices", state_indices, _i32t, (n_seq,))
    hp = _maybe(dev, "has_initial_state", has_initial_state, _i32t, (n_seq,))
    tp = _maybe(dev, "status", status, _i32t, (1,))
    out, op, os = _out(dev, v, out, (T, H, P))
    head = (qp, qs[0], qs[1], kp, ks[0], ks[1], vp, vs[0], vs[1], ap, as_[0], bp, bs[0], Ap, tb, up, ip, hp, sp, ss, op, os[0], os[1])
    tail = (tp, T, n_seq, H, P, K, G, S, _scale(scale, K), 1 if qk_norm else 0, SCAN_ROUTES[route], 0)
    wp, wn = 0, 0
    if workspace is not None:
        wn = _sizes("workspace", workspace, 1)[0]
        wp = _check(dev, "workspace", workspace, _u8, (wn,), True)
    else:
        packed = _RULE.pack(*head, 0, 0, *tail)
        if dev == torch.cuda.current_device():
            wn = _rule_workspace(packed)
        else:
            with torch.cuda.device(dev):
                wn = _rule_workspace(packed)
        if wn > 0:
            workspace = v.new_empty((wn + 1) // 2)
            wp = workspace.data_ptr()
        else:
            wn = 0  # none, or a declined call
    _RULE.launch(dev, _RULE.pack(*head, wp, wn, *tail))
    return out


def gated_delta_update(qkv, a, b, A, state, conv_state=None, conv_weight=None, conv_bias=None, activation=None, *, dt_bias=None,
                       groups=1, scale=None, qk_norm=True, state_indices=None, out=None, workspace=None, status=None):
    """One token per row: convolution step and state step of the gated delta rule, both in place on the row's slot.

    ``qkv`` BF16 ``[N, 2*G*K + H*P]`` (any row stride) holds q, then k of the ``groups`` G, then v.
    With ``conv_weight`` (BF16 ``[2*G*K + H*P, W]``) it goes through the step of
    ``causal_conv1d_update`` on ``conv_state`` (BF16 ``[S, 2*G*K + H*P, L]``) first, its result kept in
    32 bits; without, it is taken as is. Then one step of ``gated_delta_rule`` on ``state``
    (FP32 ``[S, H, P, K]``), with ``a`` and ``b`` BF16 ``[N, H]``. Returns BF16 ``[N, H, P]``. ``state_indices`` (int32
    ``[N]``) picks the slots, -1 marking padding rows (output +0). ``workspace`` (uint8, 4 bytes for every entry of
    ``qkv``) replaces the scratch the convolution otherwise takes from torch.
    """
    S, H, P, K = _sizes("state", state, 4)
    N = _sizes("qkv", qkv, 2)[0]
    channels = 2 * groups * K + H * P
    dev = qkv.get_device()
    xp = _check(dev, "qkv", qkv, _bf16, (N, channels))
    sp = _check(dev, "state", state, _f32, (S, H, P, K))
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
            workspace = qkv.new_empty(2 * N * channels)  # as BF16 entries
            ws, wn = workspace.data_ptr(), 4 * N * channels
        else:
            wn = _sizes("workspace", workspace, 1)[0]
            ws = _check(dev, "workspace", workspace, _u8, (wn,), True)
    elif conv_state is not None or conv_bias is not None:
        raise ValueError("conv_state and conv_bias need a conv_weight")
    ap = _check(dev, "a", a, _bf16, (N, H))
    bp = _check(dev, "b", b, _bf16, (N, H))
    Ap = _check(dev, "A", A, _f32, (H,), True)
    tb = _maybe(dev, "dt_bias", dt_bias, _f32, (H,))
    ip = _maybe(dev, "state_indices", state_indices, _i32t, (N,))
    tp = _maybe(dev, "status", status, _i32t, (1,))
    out, op, os = _out(dev, qkv, out, (N, H, P))
    _STEP.launch(dev, _STEP.pack(xp, _strides("qkv", qkv)[0], wp, kp, cp, *cs, ap, _strides("a", a)[0], bp, _strides("b", b)[0], Ap, tb,
                                 ip, sp, _slot_stride(state, H, P, K, "state"), op, os[0], os[1], ws, wn, tp, N, H, P, K, groups,
                                 S, L, W, _scale(scale, K), 1 if qk_norm else 0, act, 0))
    return out


def gated_rms_norm(x, z=None, weight=None, *, eps=1e-6, norm_before_gate=True, out=None):
    """The norm behind a recurrence, with its gate: ``x / rms(x) * weight * silu(z)`` over the last dimension of ``x``
    (BF16 ``[T, H, P]``, rows and heads any strides), or with ``norm_before_gate=False`` the norm of ``x * silu(z)``, times
    ``weight``. ``z`` BF16 ``[T, H, P]`` or None (no gate); ``weight`` BF16 or FP32, ``[P]`` for all heads or ``[H, P]``, or
    None; ``eps`` is added to the mean of the squares. Returns BF16 ``[T, H, P]``.
    """
    T, H, P = _sizes("x", x, 3)
    dev = x.get_device()
    xp, xs = _check(dev, "x", x, _bf16, (T, H, P)), _strides("x", x)
    zp, zs = 0, (0, 0)
    if z is not None:
        zp, zs = _check(dev, "z", z, _bf16, (T, H, P)), _strides("z", z)
    wp = wt = wh = 0
    if weight is not None:
        wt = _type("weight", weight)
        each = weight.dim() != 1
        wp, wh = _check(dev, "weight", weight, weight.dtype, (H, P) if each else (P,), True), P if each else 0
    out, op, os = _out(dev, x, out, (T, H, P))
    _GATED.launch(dev, _GATED.pack(xp, xs[0], xs[1], zp, zs[0], zs[1], wp, wh, op, os[0], os[1], T, H, P, _single(eps),
                                   0 if norm_before_gate else 1, wt, 0))
    return out


def residual_rms_norm(x, residual, weight=None, *, post_weight=None, scale=1.0, eps=1e-6, out=None):
    """Between two blocks: ``residual += scale * x`` in place, and the norm ``residual / rms(residual) * weight`` for the next
    block. With ``post_weight`` the block's output is normed too: ``residual += scale * x / rms(x) * post_weight``. ``x``
    BF16 ``[T, D]`` and ``residual`` BF16 or FP32 ``[T, D]`` (any row strides); the weights BF16 or FP32 ``[D]``, both of one
    type, ``weight`` None for ones; ``eps`` is added to the means of the squares. The norm is taken of the sum in 32 bits, which is rounded to the
    residual's type where it is stored. Returns BF16 ``[T, D]``.
    """
    T, D = _sizes("x", x, 2)
    dev = x.get_device()
    xp = _check(dev, "x", x, _bf16, (T, D))
    rt = _type("residual", residual)
    rp = _check(dev, "residual", residual, residual.dtype, (T, D))
    wp = pp = wt = 0
    if weight is not None:
        wt = _type("weight", weight)
        wp = _check(dev, "weight", weight, weight.dtype, (D,), True)
    if post_weight is not None:
        pt = _type("post_weight", post_weight)
        if weight is not None and pt != wt:
            raise ValueError(f"post_weight must be {weight.dtype} as weight is, got {post_weight.dtype}")
        wt, pp = pt, _check(dev, "post_weight", post_weight, post_weight.dtype, (D,), True)
    out, op, os = _out(dev, x, out, (T, D))
    _RESIDUAL.launch(dev, _RESIDUAL.pack(xp, _strides("x", x)[0], rp, _strides("residual", residual)[0], wp, pp, op, os[0],
                                         T, D, _single(scale), _single(eps), rt, wt))
    return out
