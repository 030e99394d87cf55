"""Buffers for results that a call does not compute, host tensors and 8-bit copies asked for by something else than a Packed are refused with a
ValueError (CPU only)."""
import pytest
import torch

import gated_delta_rule_20_amd as kda

X = torch.zeros(4, 8)
W = torch.ones(8)
P = kda.Packed(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1))


@pytest.mark.parametrize("call,name", [
    (lambda: kda.block_norm_fwd(X, X, n_out=X), "n_out without pre_weight"),
    (lambda: kda.block_norm_bwd(X, None, X, X, pre_weight=W, dy=X), "dy without y"),
    (lambda: kda.block_norm_bwd(X, X, X, X, pre_weight=W, dgate=X), "dgate without gate"),
])
def test_results_that_are_not_computed(call, name):
    with pytest.raises(ValueError, match=name):
        call()


@pytest.mark.parametrize("call", [
    lambda: kda.block_norm_fwd(X, pre_weight=W), lambda: kda.block_norm_fwd(X, pre_weight=W, n_out=X), lambda: kda.block_norm_fwd(X),
    lambda: kda.block_norm_bwd(X, None, X, X, pre_weight=W), lambda: kda.block_norm_bwd(X, None, None, X, pre_weight=W),
    lambda: kda.block_norm_bwd(None, None, X), lambda: kda.block_norm_bwd(P, None, X, X, pre_weight=W),
])
def test_host_tensors_without_a_block(call):
    with pytest.raises(ValueError, match="device tensor"):
        call()


@pytest.mark.parametrize("pack", [P, (P, P, P), [P, P, P], 1, X, "yes"])
def test_norm_copies_go_to_a_BlockNormSaved(pack):
    with pytest.raises(ValueError, match="pack must be"):
        kda.block_norm_fwd(X, X, pack=pack)


@pytest.mark.parametrize("pack", [1, X, (P.codes, P.scales), "yes"])
def test_other_copies_go_to_a_Packed(pack):
    from gated_delta_rule_20_amd.act import _packed_out
    with pytest.raises(ValueError, match="pack must be"):
        _packed_out(pack, "pack", X.shape, X.device, X.dtype)


def test_workspace_size_without_a_stream():
    with pytest.raises(ValueError, match="x_new"):
        kda.block_norm_bwd_workspace_size(None)
