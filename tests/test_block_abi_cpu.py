"""The entry points of the gated scan, the norms around a block and 8-bit activations reject bad arguments with a status before
anything is enqueued (CPU only: no call here reaches a kernel launch)."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_20_amd as kda

A = 0x10000  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_20_amd import build
        build.build()
    return kda.load_library()


def _message(lib):
    return lib.kda_last_error_message().decode()


def _set(a, over):
    for key, val in over.items():
        setattr(a, key, val)
    return a


def _fwd(**over):
    a = kda.GatedScanFwdArgs(B=2, T=300, C=96, dtype=kda.KDA_BF16, g_dtype=kda.KDA_BF16, x=A, x_stride=96, g=A, g_stride=96, h=A,
                             final_state=A, g_min=-5.0, workspace=A, workspace_bytes=1 << 30)
    return _set(a, over)


def _bwd(**over):
    a = kda.GatedScanBwdArgs(B=2, T=300, C=96, dtype=kda.KDA_BF16, g_dtype=kda.KDA_F32, g=A, g_stride=96, h=A, d_h=A, dx=A,
                             dx_stride=96, dg=A, dg_stride=96, x=A, x_stride=96, g_min=-5.0, workspace=A, workspace_bytes=1 << 30)
    return _set(a, over)


SCAN = [
    (dict(dtype=2), 1, "dtype"), (dict(dtype=-1), 1, "dtype"), (dict(g_dtype=7), 1, "g_dtype"),
    (dict(dtype=0, g_dtype=1), 2, "g_dtype"), (dict(B=0), 1, "B >= 1"), (dict(T=-1), 1, "T >= 0"), (dict(C=0), 1, "C"),
    (dict(C=(1 << 24) + 1), 1, "C"), (dict(B=1 << 15, T=1 << 17), 2, "32-bit"), (dict(B=1 << 20, T=1, C=1 << 24), 2, "too large"),
    (dict(cu_seqlens=A, N=3), 1, "B == 1"), (dict(cu_seqlens=A, B=1, N=0), 1, "N >= 1"), (dict(cu_seqlens=A + 2, B=1, N=2), 1, "cu_seqlens"),
    (dict(g=None), 1, "g is NULL"), (dict(g=A + 1), 1, "g is not"), (dict(g_stride=95), 1, "g_stride"), (dict(g_stride=-96), 1, "g_stride"),
    (dict(A_log=A + 1), 1, "A_log"), (dict(A_log=A, g_min=0.0), 1, "g_min"), (dict(A_log=A, g_min=float("nan")), 1, "g_min"),
    (dict(A_log=A, g_min=float("-inf")), 1, "g_min"), (dict(initial_state=A + 2), 1, "initial_state"),
]


@pytest.mark.parametrize("over,status,msg", SCAN + [
    (dict(x=None), 1, "x is NULL"), (dict(x=A + 1), 1, "x is not"), (dict(x_stride=95), 1, "x_stride"), (dict(x_stride=1 << 41), 1, "x_stride"),
    (dict(h=None), 1, "h is NULL"), (dict(h=A + 1), 1, "h is not"), (dict(final_state=A + 2), 1, "final_state"),
    (dict(h_codes=A), 1, "together"), (dict(h_scales=A), 1, "together"), (dict(h_codes=A, h_scales=A + 1), 1, "h is not"),
])
def test_scan_fwd_rejects(lib, over, status, msg):
    assert lib.kda_gated_scan_fwd(ctypes.byref(_fwd(**over)), None) == status
    assert msg in _message(lib)


@pytest.mark.parametrize("over,status,msg", [s for s in SCAN if s[0] != dict(dtype=0, g_dtype=1)] + [
    (dict(d_h=None), 1, "d_h is NULL"), (dict(dx=None), 1, "dx is NULL"), (dict(dx=A + 1), 1, "dx is not"), (dict(dx_stride=1), 1, "dx_stride"),
    (dict(h=None), 1, "h is NULL"), (dict(h=A + 1), 1, "h is not"), (dict(h_scales=A + 1), 1, "scales"), (dict(dg=A + 2), 1, "dg is not"),
    (dict(dg_stride=0), 1, "dg_stride"), (dict(complement=1, x=None), 1, "x is NULL"), (dict(complement=1, x_stride=0), 1, "x_stride"),
    (dict(complement=1, x_scales=A + 2), 1, "scales"), (dict(dA_log=A), 1, "A_log and dg"), (dict(dA_log=A, A_log=A, dg=None), 1, "A_log and dg"),
    (dict(dA_log=A + 2, A_log=A), 1, "dA_log"), (dict(d_final_state=A + 1), 1, "d_final_state"),
    (dict(d_initial_state=A + 1), 1, "d_initial_state"), (dict(dA_log=A, A_log=A, workspace=None), 3, "workspace"),
    (dict(dA_log=A, A_log=A, workspace_bytes=8), 3, "workspace"), (dict(dA_log=A, A_log=A, workspace=A + 128), 3, "256"),
])
def test_scan_bwd_rejects(lib, over, status, msg):
    assert lib.kda_gated_scan_bwd(ctypes.byref(_bwd(**over)), None) == status
    assert msg in _message(lib)


@pytest.mark.parametrize("over,status,msg", [
    (dict(N=-1), 1, "N >= 0"), (dict(n_slots=-1), 1, "n_slots"), (dict(slots=None, n_slots=3), 1, "at least N"), (dict(C=0), 1, "C"),
    (dict(N=1 << 30, n_slots=1 << 30), 2, "too large"), (dict(dtype=0, g_dtype=1), 2, "g_dtype"), (dict(x=None), 1, "x is NULL"),
    (dict(g=A + 1), 1, "g is not"), (dict(x_stride=3), 1, "x_stride"), (dict(g_stride=3), 1, "g_stride"), (dict(state=None), 1, "state"),
    (dict(new_state=None), 1, "new_state"), (dict(new_state=0x1000000 + 8 * 96 * 4 - 4), 1, "overlaps"), (dict(new_state=0x1000000 - 4), 1, "overlaps"),
    (dict(h=None), 1, "h is NULL"), (dict(slots=A + 2), 1, "slots"), (dict(A_log=A, g_min=1.0), 1, "g_min"),
])
def test_scan_step_rejects(lib, over, status, msg):
    a = kda.GatedScanStepArgs(N=4, C=96, dtype=kda.KDA_BF16, g_dtype=kda.KDA_BF16, x=A, x_stride=96, g=A, g_stride=96, slots=A, n_slots=8,
                              state=0x1000000, new_state=0x1000000, h=A, g_min=-5.0)
    assert lib.kda_gated_scan_step(ctypes.byref(_set(a, over)), None) == status
    assert msg in _message(lib)


NORM = [
    (dict(R=-1), 1, "R >= 0"), (dict(R=0x7fffffff), 2, "too many rows"),
    (dict(D=0), 1, "D >= 1"), (dict(D=16385), 2, "at most"), (dict(dtype=3), 1, "dtype"),
    (dict(dtype=0, x_dtype=1), 2, "x_dtype"), (dict(eps=-1e-6), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(scale=float("inf")), 1, "scale"), (dict(y=None), 1, "belong to y"), (dict(post_weight=A + 2), 1, "post_weight"),
    (dict(res_scale=A + 1), 1, "res_scale"), (dict(pre_weight=A + 2), 1, "pre_weight"), (dict(y=A + 1), 1, "y is not"),
    (dict(y_stride=4), 1, "y_stride"), (dict(gate=A + 1), 1, "gate is not"), (dict(gate_stride=4), 1, "gate_stride"),
]


@pytest.mark.parametrize("over,status,msg", NORM + [
    (dict(y=None, gate=None, post_weight=None, res_scale=None, pre_weight=None), 1, "nothing"), (dict(x=None), 1, "x is NULL"),
    (dict(x=A + 2), 1, "x is not"), (dict(x_out=None), 1, "x_out is NULL"), (dict(x_out=0x1000000 + 4), 1, "overlaps"), (dict(n=None), 1, "n is NULL"),
    (dict(x_codes=A), 1, "together"), (dict(y_scales=A), 1, "together"), (dict(gate=None, gate_codes=A, gate_scales=A), 1, "without it"),
])
def test_norm_fwd_rejects(lib, over, status, msg):
    a = kda.BlockNormFwdArgs(R=7, D=96, dtype=kda.KDA_BF16, x_dtype=kda.KDA_F32, x=0x1000000, y=A, y_stride=96, gate=A, gate_stride=96, post_weight=A,
                             res_scale=A, pre_weight=A, scale=1.0, eps=1e-6, x_out=0x2000000, n=A)
    assert lib.kda_block_norm_fwd(ctypes.byref(_set(a, over)), None) == status
    assert msg in _message(lib)


@pytest.mark.parametrize("over,status,msg", NORM + [
    (dict(d_x_new=None, d_n=None), 1, "neither"), (dict(pre_weight=None), 1, "without"), (dict(post_weight=None), 1, "without the weight"),
    (dict(dx=None), 1, "dx is NULL"), (dict(dx=0x1000000 + 4), 1, "overlaps"), (dict(x_new=None), 1, "x_new is NULL"),
    (dict(x_scales=A + 2), 1, "scales"), (dict(d_n=A + 1), 1, "d_n"), (dict(d_x_new=0x1000002), 1, "d_x_new"), (dict(dy=None), 1, "dy is NULL"),
    (dict(dy_stride=4), 1, "dy_stride"), (dict(dgate=None), 1, "dgate is NULL"), (dict(dgate_stride=4), 1, "dgate_stride"),
    (dict(d_pre_weight=A + 2), 1, "d_pre_weight"), (dict(workspace=None), 3, "workspace"), (dict(workspace_bytes=100), 3, "workspace"),
])
def test_norm_bwd_rejects(lib, over, status, msg):
    a = kda.BlockNormBwdArgs(R=7, D=96, dtype=kda.KDA_BF16, x_dtype=kda.KDA_F32, x_new=A, y=A, y_stride=96, gate=A, gate_stride=96, post_weight=A,
                             res_scale=A, pre_weight=A, scale=1.0, eps=1e-6, d_x_new=0x1000000, d_n=A, dx=0x2000000, dy=A, dy_stride=96, dgate=A,
                             dgate_stride=96, d_post_weight=A, d_res_scale=A, d_pre_weight=A, workspace=A, workspace_bytes=1 << 30)
    assert lib.kda_block_norm_bwd(ctypes.byref(_set(a, over)), None) == status
    assert msg in _message(lib)


@pytest.mark.parametrize("args,status,msg", [
    ((2, A, 8, 4, 8, A, A, None), 1, "dtype"), ((1, A, 8, -1, 8, A, A, None), 1, "R >= 0"), ((1, A, 8, 4, 0, A, A, None), 1, "D >= 1"),
    ((1, A, 7, 4, 8, A, A, None), 1, "x_stride"), ((1, None, 8, 4, 8, A, A, None), 1, "x is NULL"), ((1, A + 1, 8, 4, 8, A, A, None), 1, "x is not"),
    ((1, A, 8, 4, 8, None, A, None), 1, "codes"), ((1, A, 8, 4, 8, A, A + 1, None), 1, "scales"),
    ((1, A, 1 << 20, 1 << 40, 1 << 20, A, A, None), 2, "too large"),
])
def test_act_pack_rejects(lib, args, status, msg):
    assert lib.kda_act_pack(*args) == status
    assert msg in _message(lib)
    dtype, x, _, R, D, codes, scales, s = args
    if msg != "x_stride":
        assert lib.kda_act_unpack(dtype, codes, scales, R, D, x, s) == status
        assert msg in _message(lib)


def test_null_and_empty(lib):
    for fn in ("kda_gated_scan_fwd", "kda_gated_scan_bwd", "kda_gated_scan_step", "kda_block_norm_fwd", "kda_block_norm_bwd"):
        assert getattr(lib, fn)(None, None) == 1
    n = ctypes.c_size_t(0)
    for fn, a in (("kda_gated_scan_fwd", _fwd()), ("kda_gated_scan_bwd", _bwd())):
        assert getattr(lib, fn + "_workspace_size")(None, ctypes.byref(n)) == 1
        assert getattr(lib, fn + "_workspace_size")(ctypes.byref(a), None) == 1
    assert lib.kda_gated_scan_fwd(ctypes.byref(_fwd(T=0, x=None, g=None, h=None, final_state=None)), None) == 0
    assert lib.kda_gated_scan_step(ctypes.byref(kda.GatedScanStepArgs(N=0, C=8, n_slots=0)), None) == 0
    assert lib.kda_block_norm_fwd(ctypes.byref(kda.BlockNormFwdArgs(R=0, D=8, scale=1.0)), None) == 0
    assert lib.kda_block_norm_bwd(ctypes.byref(kda.BlockNormBwdArgs(R=0, D=8, scale=1.0)), None) == 0
    assert lib.kda_act_pack(1, None, 0, 0, 8, None, None, None) == 0
    assert lib.kda_act_unpack(1, None, None, 0, 8, None, None) == 0


def test_python_refuses_host_tensors():
    x = torch.zeros(1, 4, 8)
    for call in (lambda: kda.gated_scan_fwd(x, x), lambda: kda.gated_scan_bwd(None, x, x, x), lambda: kda.gated_scan_fwd(None, x),
                 lambda: kda.gated_scan_step(x[0], x[0], x[0]), lambda: kda.block_norm_fwd(x, x), lambda: kda.block_norm_fwd(None),
                 lambda: kda.block_norm_bwd(x, x, x), lambda: kda.block_norm_bwd(x, x, None, None), lambda: kda.act_pack(x),
                 lambda: kda.act_pack(None), lambda: kda.act_unpack(x), lambda: kda.act_unpack(kda.Packed(None, None)),
                 lambda: kda.act_unpack(kda.Packed(x.to(torch.int8), x)), lambda: kda.gated_scan_fwd(x.half(), x.half())):
        with pytest.raises(ValueError):
            call()
