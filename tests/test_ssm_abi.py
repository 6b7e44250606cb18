"""The state-space operators' argument checks, without a GPU: every decline happens before any
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

CONV = dict(x=A16, ld_x=64, weight=A16, conv_state=A16, stride_s=192, stride_d=1, stride_l=64, cu_seqlens=A16, out=A16,
            ld_out=64, T=10, B=2, D=64, S=4, L=3, W=4)
SCAN = dict(x=A16, x_stride_t=128, x_stride_h=64, dt=A16, dt_stride_t=2, b=A16, b_stride_t=128, b_stride_g=128, c=A16,
            c_stride_t=128, c_stride_g=128, A=A16, cu_seqlens=A16, state=A16, state_stride_s=2 * 64 * 128, out=A16,
            out_stride_t=128, out_stride_h=64, workspace=A16, workspace_bytes=1 << 40, T=10, n_seq=2, H=2, P=64, K=128, G=1,
            S=4, dt_softplus=1)
STEP = dict(xbc=A16, ld_xbc=384, conv_weight=A16, conv_state=A16, conv_stride_s=384 * 3, conv_stride_d=3, conv_stride_l=1,
            dt=A16, dt_stride_n=2, A=A16, state=A16, state_stride_s=2 * 64 * 128, out=A16, out_stride_n=128, out_stride_h=64,
            workspace=A16, workspace_bytes=1 << 40, N=3, H=2, P=64, K=128, G=1, S=4, L=3, W=4, dt_softplus=1)
W4 = dict(x=A16, ld_x=256, qweight=A16, scales=A16, out=A16, ld_out=32, M=3, I=256, O=32, group=128)

DECLINES = [
    ("causal_conv1d_packed", CONV, [
        (dict(act=2), 1, "act"), (dict(T=-1), 1, ">= 0"), (dict(W=0), 1, "W must be"), (dict(W=5), 2, "widths 2 to 4"),
        (dict(T=1 << 31), 2, "2^31"), (dict(cu_seqlens=None), 1, "cu_seqlens"), (dict(weight=None), 1, "NULL"),
        (dict(out=None), 1, "NULL"), (dict(x=A16 + 1), 1, "2-byte"), (dict(indices=A16 + 2), 1, "4-byte"),
        (dict(ld_x=63), 1, "row strides"), (dict(ld_out=1), 1, "row strides"), (dict(L=2), 1, "L must be >= W - 1"),
        (dict(S=1), 1, "S must be >= B"), (dict(conv_state=None, has_initial=A16), 1, "need a conv_state"),
        (dict(stride_l=-1), 1, "strides"), (dict(ld_x=1 << 61), 1, "overflow"), (dict(S=1 << 60, indices=A16), 1, "overflow")]),
    ("selective_scan", SCAN, [
        (dict(H=3, G=2), 1, "multiple of G"), (dict(G=0), 1, "multiple of G"), (dict(K=0), 1, "K must be >= 1"),
        (dict(K=257), 2, "K <= 256"), (dict(n_seq=-1), 1, ">= 0"), (dict(route=3), 1, "unknown route"), (dict(route=-1), 1, "unknown route"),
        (dict(T=1 << 31), 2, "2^31"), (dict(A=None), 1, "A must"), (dict(dt=None), 1, "NULL"), (dict(cu_seqlens=None), 1, "cu_seqlens"),
        (dict(z=A16 + 1), 1, "2-byte"), (dict(D=A16 + 2), 1, "FP32"), (dict(has_initial=A16 + 1), 1, "4-byte"),
        (dict(workspace=A16 + 8), 1, "workspace"), (dict(b_stride_g=-1), 1, "strides"), (dict(S=1), 1, "S must be >= n_seq"),
        (dict(state=None), 1, "state must not be NULL"), (dict(state_stride_s=100), 1, "overlap"),
        (dict(x_stride_t=1 << 60), 1, "overflow"), (dict(n_seq=1 << 30, S=1 << 30), 2, "2^31"), (dict(P=1 << 56), 1, "overflow")]),
    ("selective_state_update", STEP, [
        (dict(act=7), 1, "act"), (dict(N=-1), 1, "N must"), (dict(W=0), 1, "W must"), (dict(L=2), 1, "L must be >= W - 1"),
        (dict(W=1, L=0), 2, "empty state"), (dict(ld_xbc=383), 1, "ld_xbc"), (dict(K=300, ld_xbc=1000), 2, "K <= 256"),
        (dict(xbc=None), 1, "NULL"), (dict(conv_state=None), 1, "conv_state"), (dict(conv_stride_d=-1), 1, "strides"),
        (dict(workspace=None), 1, "workspace"), (dict(workspace_bytes=3 * 384 * 4 - 1), 1, "workspace"),
        (dict(S=2), 1, "S must be >= N"), (dict(out=A16 + 1), 1, "2-byte"), (dict(indices=A16 + 1), 1, "4-byte"),
        (dict(H=5, G=2, ld_xbc=10000), 1, "multiple of G"), (dict(z_stride_h=-8), 1, "strides"),
        (dict(N=1 << 30, S=1 << 30, conv_weight=None, state_stride_s=2 * 64 * 128), 2, "2^31")]),
    ("w4_matmul", W4, [
        (dict(M=-1), 1, ">= 0"), (dict(group=0), 1, "group"), (dict(group=16), 2, "groups of"), (dict(I=200, ld_x=200), 1, "multiple of group"),
        (dict(x=None), 1, "NULL"), (dict(scales=None), 1, "NULL"), (dict(out=None), 1, "NULL"), (dict(zeros=A16 + 1), 1, "2-byte"),
        (dict(qweight=A16 + 2), 1, "4-byte"), (dict(ld_x=255), 1, "row strides"), (dict(ld_out=31), 1, "row strides"),
        (dict(O=1 << 60, M=1), 1, "overflow")]),
]
STRUCTS = {"causal_conv1d_packed": "Conv1dPackedArgs", "selective_scan": "SelectiveScanArgs",
           "selective_state_update": "SelectiveStateUpdateArgs", "w4_matmul": "W4MatmulArgs"}


@pytest.mark.parametrize("op,base,change,status,message",
                         [(op, base, *d) for op, base, ds in DECLINES for d in ds],
                         ids=lambda v: str(v) if isinstance(v, (str, int)) else None)
def test_decline(ccu, op, base, change, status, message):
    args = getattr(ccu, STRUCTS[op])(**{**base, **change})
    assert getattr(ccu, "ccu_" + op)(args, None) == status
    assert message in ccu.ccu_conv1d_last_error()
    if op == "selective_scan":
        assert ccu.ccu_selective_scan_select_route(args) == -1


def test_null_args(ccu):
    for op in STRUCTS:
        assert getattr(ccu.lib, "ccu_" + op)(None, None) == 1
        assert "args" in ccu.ccu_conv1d_last_error()
    assert ccu.lib.ccu_selective_scan_workspace_bytes(None) == -1


def test_nothing_to_do(ccu):
    for op, base, none in (("causal_conv1d_packed", CONV, dict(D=0)), ("causal_conv1d_packed", CONV, dict(B=0)),
                           ("selective_scan", SCAN, dict(n_seq=0)), ("selective_scan", SCAN, dict(H=0)),
                           ("selective_state_update", STEP, dict(N=0)), ("selective_state_update", STEP, dict(P=0)),
                           ("w4_matmul", W4, dict(M=0)), ("w4_matmul", W4, dict(O=0))):
        assert getattr(ccu, "ccu_" + op)(getattr(ccu, STRUCTS[op])(**{**base, **none}), None) == 0


def test_workspace_bytes(ccu):
    assert ccu.ccu_selective_state_update_workspace_bytes(3, 2, 64, 128, 1, 1) == 3 * 384 * 4
    assert ccu.ccu_selective_state_update_workspace_bytes(3, 2, 64, 128, 1, 0) == 0
    assert ccu.ccu_selective_state_update_workspace_bytes(-1, 2, 64, 128, 1, 1) == -1
    assert ccu.ccu_selective_scan_workspace_bytes(ccu.SelectiveScanArgs(**SCAN)) >= 0


def test_structs_match_the_header(ccu, tmp_path):
    """Sizes and the offsets of the last members, as a C compiler lays them out."""
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"ccu_conv1d_packed_args_t": (ccu.Conv1dPackedArgs, "reserved"), "ccu_selective_scan_args_t": (ccu.SelectiveScanArgs, "route"),
             "ccu_selective_state_update_args_t": (ccu.SelectiveStateUpdateArgs, "dt_softplus"), "ccu_w4_matmul_args_t": (ccu.W4MatmulArgs, "group")}
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
    x, w = torch.zeros(4, 8, dtype=bf), torch.zeros(8, 4, dtype=bf)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        ccu.causal_conv1d_packed([1.0], w, cu_seqlens=None)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ccu.causal_conv1d_packed(x, w, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="activation"):
        ccu.causal_conv1d_packed(x, w, None, "relu", cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="x must be torch.bfloat16"):
        ccu.selective_scan(torch.zeros(4, 2, 8), None, None, None, None, cu_seqlens=None, ssm_state=None)
    with pytest.raises(ValueError, match="route"):
        ccu.selective_scan(x, None, None, None, None, cu_seqlens=None, ssm_state=None, route="bulk")
    with pytest.raises(ValueError, match="ssm_state must have 4 dimensions"):
        ccu.selective_state_update(x, x, None, torch.zeros(1, 4, 2, dtype=bf))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ccu.w4_matmul(x, torch.zeros(3, 4, dtype=torch.uint8), torch.zeros(3, 1, dtype=bf))
    with pytest.raises(ValueError, match="multiple of group"):
        ccu.w4_quantize(torch.zeros(4, 100, dtype=f), 64)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_takes_a_parameter(ccu, symmetric):
    """A module's weight requires grad; its 4-bit form does not (w4_matmul refuses scales that do)."""
    import torch

    w = torch.nn.Parameter(torch.randn(4, 128))
    got = ccu.w4_quantize(w, 64, symmetric)
    assert not any(v.requires_grad for v in got if v is not None)
    assert all(torch.equal(a, b) for a, b in zip(got, ccu.w4_quantize(w.detach(), 64, symmetric)) if a is not None)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_of_weights_below_the_scales_range(ccu, symmetric):
    """A group whose scale would round to zero in BF16 is a group of zeros, not of NaN."""
    import torch

    q, s, z = ccu.w4_quantize(torch.rand(2, 64) * 1e-41, 64, symmetric)
    assert (s > 0).all() and (z is None or z.isfinite().all())
    zero = 8 if z is None else z.float()
    assert ((q & 15) == zero).all() and ((q >> 4) == zero).all()


def test_package_imports_without_torch(ccu):
    """The raw calls need no PyTorch: the package imports without it, and takes it in at the first torch-level operator."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import sys
sys.modules["torch"] = None   # an import of it raises
import depthwise_causal_conv1d_gb300 as ccu
assert ccu.ccu_w4_matmul(ccu.W4MatmulArgs(M=-1, group=128), None) == 1 and "M, I and O" in ccu.ccu_conv1d_last_error()
assert ccu.SCAN_ROUTES["chunked"] == 2 and "selective_scan" in dir(ccu) and not hasattr(ccu, "no_such_name")
del sys.modules["torch"]
import torch
from depthwise_causal_conv1d_gb300 import selective_scan, w4_quantize
assert callable(ccu.w4_matmul) and ccu.selective_scan is selective_scan
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
