"""The argument checks of the gated delta rule and of the norms around a layer, without a GPU: every decline happens before any
CUDA call, and the message says what is wrong."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ccu():
    import __graft_entry__ as g

    g.build()
    import depthwise_causal_conv1d_gb300 as ccu

    return ccu


A16 = 0x100000  # an aligned address, never dereferenced: every call here is declined
INF, NAN = float("inf"), float("nan")

RULE = dict(q=A16, q_stride_t=128, q_stride_g=128, k=A16, k_stride_t=128, k_stride_g=128, v=A16, v_stride_t=128, v_stride_h=64,
            a=A16, a_stride_t=2, b=A16, b_stride_t=2, A=A16, cu_seqlens=A16, state=A16, state_stride_s=2 * 64 * 128, out=A16,
            out_stride_t=128, out_stride_h=64, workspace=A16, workspace_bytes=1 << 40, T=10, n_seq=2, H=2, P=64, K=128, G=1, S=4,
            qk_norm=1)
STEP = dict(qkv=A16, ld_qkv=384, conv_weight=A16, conv_state=A16, conv_stride_s=384 * 3, conv_stride_d=3, conv_stride_l=1, a=A16,
            a_stride_n=2, b=A16, b_stride_n=2, A=A16, state=A16, state_stride_s=2 * 64 * 128, out=A16, out_stride_n=128,
            out_stride_h=64, workspace=A16, workspace_bytes=1 << 40, N=3, H=2, P=64, K=128, G=1, S=4, L=3, W=4, qk_norm=1)
GATED = dict(x=A16, x_stride_t=128, x_stride_h=64, z=A16, z_stride_t=128, z_stride_h=64, weight=A16, out=A16, out_stride_t=128,
             out_stride_h=64, T=5, H=2, P=64, eps=1e-6)
RESIDUAL = dict(x=A16, ld_x=64, residual=A16, ld_residual=64, weight=A16, out=A16, ld_out=64, T=5, D=64, scale=1.0, eps=1e-6)

DECLINES = [
    ("gated_delta_rule", RULE, [
        (dict(H=3, G=2), 1, "multiple of G"), (dict(G=0), 1, "multiple of G"), (dict(K=0), 1, "K must be >= 1"),
        (dict(K=257), 2, "K <= 256"), (dict(n_seq=-1), 1, ">= 0"), (dict(route=3), 1, "unknown route"), (dict(route=-1), 1, "unknown route"),
        (dict(T=1 << 31), 2, "2^31"), (dict(A=None), 1, "A must"), (dict(a=None), 1, "NULL"), (dict(b=None), 1, "NULL"),
        (dict(q=None), 1, "NULL"), (dict(cu_seqlens=None), 1, "cu_seqlens"), (dict(v=A16 + 1), 1, "2-byte"),
        (dict(dt_bias=A16 + 2), 1, "FP32"), (dict(has_initial=A16 + 1), 1, "4-byte"), (dict(workspace=A16 + 8), 1, "workspace"),
        (dict(k_stride_g=-1), 1, "strides"), (dict(S=1), 1, "S must be >= n_seq"), (dict(state=None), 1, "state must not be NULL"),
        (dict(state_stride_s=100), 1, "overlap"), (dict(v_stride_t=1 << 60), 1, "overflow"), (dict(scale=INF), 1, "scale"),
        (dict(scale=NAN), 1, "scale"), (dict(n_seq=1 << 30, S=1 << 30), 2, "2^31"), (dict(P=1 << 56), 1, "overflow")]),
    ("gated_delta_update", STEP, [
        (dict(act=7), 1, "act"), (dict(N=-1), 1, "N must"), (dict(W=0), 1, "W must"), (dict(L=2), 1, "L must be >= W - 1"),
        (dict(W=1, L=0), 2, "empty state"), (dict(ld_qkv=383), 1, "ld_qkv"), (dict(K=300, ld_qkv=1000), 2, "K <= 256"),
        (dict(qkv=None), 1, "NULL"), (dict(b=None), 1, "NULL"), (dict(conv_state=None), 1, "conv_state"),
        (dict(conv_stride_d=-1), 1, "strides"), (dict(workspace=None), 1, "workspace"),
        (dict(workspace_bytes=3 * 384 * 4 - 1), 1, "workspace"), (dict(S=2), 1, "S must be >= N"), (dict(out=A16 + 1), 1, "2-byte"),
        (dict(indices=A16 + 1), 1, "4-byte"), (dict(H=5, G=2, ld_qkv=10000), 1, "multiple of G"), (dict(a_stride_n=-8), 1, "strides"),
        (dict(scale=-INF), 1, "scale"), (dict(N=1 << 30, S=1 << 30, conv_weight=None), 2, "2^31")]),
    ("gated_rms_norm", GATED, [
        (dict(T=-1), 1, ">= 0"), (dict(weight_type=2), 1, "type"), (dict(eps=-1.0), 1, "eps"), (dict(eps=NAN), 1, "eps"),
        (dict(eps=INF), 1, "eps"), (dict(x=None), 1, "NULL"), (dict(out=None), 1, "NULL"), (dict(z=A16 + 1), 1, "2-byte"),
        (dict(weight=A16 + 2, weight_type=1), 1, "weight"), (dict(out_stride_h=-1), 1, "strides"), (dict(weight_stride_h=-1), 1, "strides"),
        (dict(x_stride_t=1 << 61), 1, "overflow"), (dict(T=1 << 31, H=1), 2, "2^31")]),
    ("residual_rms_norm", RESIDUAL, [
        (dict(D=-1), 1, ">= 0"), (dict(weight_type=-1), 1, "type"), (dict(residual_type=3), 1, "type"), (dict(eps=-1.0), 1, "eps"),
        (dict(scale=NAN), 1, "scale"), (dict(x=None), 1, "NULL"), (dict(residual=None), 1, "NULL"), (dict(out=None), 1, "NULL"),
        (dict(out=A16 + 1), 1, "2-byte"), (dict(residual=A16 + 2, residual_type=1), 1, "residual"),
        (dict(post_weight=A16 + 1), 1, "weights"), (dict(ld_residual=63), 1, "row strides"), (dict(ld_out=0), 1, "row strides"),
        (dict(ld_x=1 << 61), 1, "overflow"), (dict(T=1 << 31), 2, "2^31")]),
]
STRUCTS = {"gated_delta_rule": "GatedDeltaRuleArgs", "gated_delta_update": "GatedDeltaUpdateArgs", "gated_rms_norm": "GatedRmsNormArgs",
           "residual_rms_norm": "ResidualRmsNormArgs"}


@pytest.mark.parametrize("op,base,change,status,message",
                         [(op, base, *d) for op, base, ds in DECLINES for d in ds],
                         ids=lambda v: str(v) if isinstance(v, (str, int)) else None)
def test_decline(ccu, op, base, change, status, message):
    args = getattr(ccu, STRUCTS[op])(**{**base, **change})
    assert getattr(ccu, "ccu_" + op)(args, None) == status
    assert message in ccu.ccu_conv1d_last_error()
    if op == "gated_delta_rule":
        assert ccu.ccu_gated_delta_rule_select_route(args) == -1
        assert ccu.ccu_gated_delta_rule_workspace_bytes(args) == -1


def test_route(ccu):
    """AUTO takes the chunked kernel where it serves and the sequences are long enough on average."""
    route = lambda **kw: ccu.ccu_gated_delta_rule_select_route(ccu.GatedDeltaRuleArgs(**{**RULE, **kw}))  # noqa: E731
    auto, recurrent, chunked = 0, 1, 2
    long = dict(T=2000, n_seq=2)
    assert route(**long) == chunked and route(T=63) == recurrent and route(T=64) == chunked and route(T=3, route=chunked) == chunked
    wide = dict(P=128, v_stride_t=256, v_stride_h=128, out_stride_t=256, out_stride_h=128, state_stride_s=2 * 128 * 128)
    assert route(T=31, **wide) == recurrent and route(T=32, **wide) == chunked
    assert route(**long, route=recurrent) == recurrent and route(n_seq=0) == auto
    for kw in (dict(K=136, state_stride_s=2 * 64 * 136), dict(K=100), dict(P=60), dict(q=A16 + 2), dict(k_stride_t=100), dict(v_stride_h=0), dict(v_stride_t=1 << 40),
               dict(out=A16 + 2), dict(out_stride_t=132), dict(state=A16 + 4), dict(state_stride_s=2 * 64 * 128 + 2)):
        assert route(**long, **kw) == recurrent
        assert route(**long, **kw, route=chunked) == -1 and "chunked delta rule" in ccu.ccu_conv1d_last_error()


def test_null_args(ccu):
    for op in STRUCTS:
        assert getattr(ccu.lib, "ccu_" + op)(None, None) == 1
        assert "args" in ccu.ccu_conv1d_last_error()
    assert ccu.lib.ccu_gated_delta_rule_workspace_bytes(None) == -1


def test_nothing_to_do(ccu):
    for op, base, none in (("gated_delta_rule", RULE, dict(n_seq=0)), ("gated_delta_rule", RULE, dict(H=0)),
                           ("gated_delta_rule", RULE, dict(P=0)), ("gated_delta_update", STEP, dict(N=0)),
                           ("gated_delta_update", STEP, dict(P=0)), ("gated_rms_norm", GATED, dict(T=0)),
                           ("gated_rms_norm", GATED, dict(P=0)), ("residual_rms_norm", RESIDUAL, dict(T=0)),
                           ("residual_rms_norm", RESIDUAL, dict(D=0))):
        assert getattr(ccu, "ccu_" + op)(getattr(ccu, STRUCTS[op])(**{**base, **none}), None) == 0


def test_workspace_bytes(ccu):
    assert ccu.ccu_gated_delta_update_workspace_bytes(3, 2, 64, 128, 1, 1) == 3 * 384 * 4
    assert ccu.ccu_gated_delta_update_workspace_bytes(3, 2, 64, 128, 1, 0) == 0
    assert ccu.ccu_gated_delta_update_workspace_bytes(-1, 2, 64, 128, 1, 1) == -1
    assert ccu.ccu_gated_delta_rule_workspace_bytes(ccu.GatedDeltaRuleArgs(**RULE)) >= 0


def test_structs_match_the_header(ccu, tmp_path):
    """Sizes and the offsets of the last members, as a C compiler lays them out."""
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"ccu_gated_delta_rule_args_t": (ccu.GatedDeltaRuleArgs, "reserved"),
             "ccu_gated_delta_update_args_t": (ccu.GatedDeltaUpdateArgs, "reserved"),
             "ccu_gated_rms_norm_args_t": (ccu.GatedRmsNormArgs, "reserved"),
             "ccu_residual_rms_norm_args_t": (ccu.ResidualRmsNormArgs, "weight_type")}
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ccu_ssm.h"\nint main(void){' + "".join(
        f'printf("%zu %zu\\n", sizeof({c}), offsetof({c}, {last}));' for c, (_, last) in names.items()) + "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, line.split())) for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()]
    assert got == [(ctypes.sizeof(s), getattr(s, last).offset) for s, last in names.values()]


def test_torch_level_refusals(ccu):
    """CPU tensors, wrong types and shapes are refused by name before anything else."""
    import torch

    bf, f = torch.bfloat16, torch.float32
    x, w = torch.zeros(4, 8, dtype=bf), torch.zeros(8, dtype=bf)
    v = torch.zeros(4, 2, 8, dtype=bf)
    with pytest.raises(TypeError, match="v must be a torch.Tensor"):
        ccu.gated_delta_rule(v, v, [1.0], x, x, None, cu_seqlens=None, state=None)
    with pytest.raises(ValueError, match="v must be a CUDA tensor"):
        ccu.gated_delta_rule(v, v, v, x, x, None, cu_seqlens=None, state=None)
    with pytest.raises(ValueError, match="v must be torch.bfloat16"):
        ccu.gated_delta_rule(v, v, v.float(), x, x, None, cu_seqlens=None, state=None)
    with pytest.raises(ValueError, match="route"):
        ccu.gated_delta_rule(v, v, v, x, x, None, cu_seqlens=None, state=None, route="bulk")
    with pytest.raises(ValueError, match="state must have 4 dimensions"):
        ccu.gated_delta_update(x, x, x, None, torch.zeros(1, 4, 2))
    with pytest.raises(ValueError, match="qkv must be a CUDA tensor"):
        ccu.gated_delta_update(x, x, x, None, torch.zeros(4, 1, 4, 16))
    with pytest.raises(ValueError, match="x must have 3 dimensions"):
        ccu.gated_rms_norm(x)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ccu.gated_rms_norm(v, v, w)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ccu.residual_rms_norm(x, x.to(f), w)
    from depthwise_causal_conv1d_gb300 import delta

    for bad in (0.0, INF, NAN):
        with pytest.raises(ValueError, match="scale"):
            delta._scale(bad, 64)
    assert delta._scale(None, 64) == 0.125 and delta._scale(-2.0, 64) == -2.0
    with pytest.raises(ValueError, match="weight must be torch.bfloat16 or torch.float32"):
        delta._type("weight", torch.zeros(8, dtype=torch.float16))


def test_names(ccu):
    """The torch-level calls are names of the package, imported at their first use."""
    for name in ("gated_delta_rule", "gated_delta_update", "gated_rms_norm", "residual_rms_norm"):
        assert name in dir(ccu) and callable(getattr(ccu, name))
