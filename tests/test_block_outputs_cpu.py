"""Buffers for results that a call does not compute, and 8-bit copies asked for by something else than a Packed, are refused with a
ValueError before anything else is looked at (CPU only)."""
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
