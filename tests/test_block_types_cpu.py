"""Which types block_norm_bwd takes its blocks and its residual stream to have, and what a Packed knows of its own (CPU only)."""
import copy
import itertools
import pickle

import pytest
import torch

import gated_delta_rule_20_amd as kda
from gated_delta_rule_20_amd.block import _types

BF, FP = torch.bfloat16, torch.float32
NAMES = ("x_new", "y", "gate", "dx_new", "dn", "dtype", "dx", "dy", "dgate")


def _pick(**given):
    return _types(*(given.get(k) for k in NAMES))


def _tensor(dtype):
    return torch.zeros(2, 4, dtype=dtype)


def _packed(dtype):
    return kda.Packed(torch.zeros(2, 4, dtype=torch.int8), torch.zeros(2, 1), dtype)


def test_packed_is_a_pair_with_a_type():
    p = _packed(BF)
    codes, scales = p
    assert codes is p.codes and scales is p.scales and len(p) == 2 and p.dtype is BF and p.shape == (2, 4)
    assert kda.Packed(codes, scales).dtype is None and kda.Packed(codes, scales, dtype=FP).dtype is FP
    assert copy.copy(p).dtype is BF and copy.deepcopy(p).dtype is BF and pickle.loads(pickle.dumps(p)).dtype is BF
    assert p._replace(scales=scales).dtype is BF
    with pytest.raises(ValueError, match="dtype"):
        kda.Packed(codes, scales, torch.float16)


@pytest.mark.parametrize("types", [(FP, FP), (BF, BF), (BF, FP)])
def test_any_tensor_or_typed_packed_names_its_type(types):
    dtype, x_dtype = types
    for make_x, make_b in itertools.product((_tensor, _packed), repeat=2):
        for x_name in ("x_new", "dx_new", "dx"):
            for b_name in ("y", "gate", "dn", "dy", "dgate"):
                if (make_x is _packed and x_name != "x_new") or (make_b is _packed and b_name not in ("y", "gate")):
                    continue
                given = {"y": _packed(None), x_name: make_x(x_dtype), b_name: make_b(dtype)}
                assert _pick(**given) == (dtype, x_dtype), given
    assert _pick(dx_new=_tensor(x_dtype), y=_packed(None), dtype=dtype) == (dtype, x_dtype)


def test_what_no_argument_names_is_refused():
    for given in (dict(dx_new=_tensor(FP), y=_packed(None)), dict(dx_new=_tensor(FP), y=_packed(None), gate=_packed(None))):
        with pytest.raises(ValueError, match="blocks' dtype"):
            _pick(**given)
    for given in (dict(dn=_tensor(BF), x_new=_packed(None)), dict(dn=_tensor(BF), x_new=_packed(None), dtype=BF)):
        with pytest.raises(ValueError, match="residual stream's dtype"):
            _pick(**given)
    # one type settles the other
    assert _pick(dx_new=_tensor(BF), y=_packed(None)) == (BF, BF)
    assert _pick(dn=_tensor(FP), x_new=_packed(None)) == (FP, FP)
    # without blocks there is no type of theirs to know
    assert _pick(dx_new=_tensor(FP)) == (FP, FP)
    # tensors, which a call checks, come before what a Packed says
    assert _pick(dn=_tensor(BF), y=_packed(FP), x_new=_packed(BF), dx=_tensor(FP)) == (BF, FP)
    with pytest.raises(ValueError, match="unsupported"):
        _pick(dx_new=_tensor(torch.float16), dn=_tensor(torch.float16))
