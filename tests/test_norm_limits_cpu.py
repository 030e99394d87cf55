"""The norms' gradients plan sums of at most 64 rows a side, whatever the rows, and refuse what no launch holds (CPU only)."""
import ctypes

import pytest
import torch

import gated_delta_rule_20_amd as kda


def _bytes(R, D, dtype):
    n = ctypes.c_size_t(0)
    a = kda.BlockNormBwdArgs(R=R, D=D, dtype=dtype, x_dtype=dtype, scale=1.0, eps=1e-6, d_pre_weight=16)
    return kda.load_library().kda_block_norm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)), n.value


@pytest.mark.parametrize("D,side,numbers", [(70, 4, 0), (500, 2, 0), (1000, 1, 0), (2000, 1, 0), (4096, 1, 0), (8000, 1, 0), (8300, 1, 16),
                                            (16384, 1, 16)])
@pytest.mark.parametrize("R", [1, 63, 8192, 16385, 262145, 5000011])
def test_sums_of_few_rows(R, D, side, numbers):
    status, size = _bytes(R, D, kda.KDA_BF16)
    assert status == 0
    parts = (size - numbers * R) // (12 * D)
    assert parts * side * 64 >= R and parts <= max(1024, 2 * R // (64 * side))


def test_too_many_workgroups():
    status, _ = _bytes(0x7fff0000, 1, kda.KDA_F32)
    assert status == 0
    status, _ = _bytes(0x7fff0000, 16384, kda.KDA_BF16)
    assert status == 2 and b"too large" in kda.load_library().kda_last_error_message()


@pytest.mark.parametrize("D", [70, 4096, 4097, 5000, 6000, 7000, 8192, 8193, 16384])
@pytest.mark.parametrize("R", [7, 8192, 16385, 20000, 26177, 33000, 100003])
def test_the_size_asked_for_is_enough(R, D):
    """Whatever blocks a stream has."""
    bf, fp = _bytes(R, D, kda.KDA_BF16)[1], _bytes(R, D, kda.KDA_F32)[1]
    rows = lambda t: torch.empty(R, D, dtype=t, device="meta")  # noqa: E731
    packed = lambda t: kda.Packed(rows(torch.int8), None, t)  # noqa: E731
    assert kda.block_norm_bwd_workspace_size(rows(torch.bfloat16)) == kda.block_norm_bwd_workspace_size(packed(torch.bfloat16)) == bf
    for x in (rows(torch.float32), packed(torch.float32), packed(None)):
        assert kda.block_norm_bwd_workspace_size(x) == max(bf, fp)
