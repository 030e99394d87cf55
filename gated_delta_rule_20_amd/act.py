"""Activations kept in 8 bits (``kda_act_*``): int8 codes with one float32 scale for each 128 consecutive values of a row.

A :class:`Packed` stands in for a tensor where a backward call reads activations that the forward has kept:
``gated_scan_bwd``, ``block_norm_bwd``, ``linear_chunk_bwd``.

Every call also takes ``stream`` (a torch.cuda.Stream; None: the current one).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _DTYPES
from .linear import _call, _check_tensors, _on_stream, _required

ACT_GROUP = 128  # KDA_ACT_GROUP


class _Pair(NamedTuple):
    codes: torch.Tensor
    scales: torch.Tensor


class Packed(_Pair):
    """A tensor [..., D] in 8 bits: ``codes`` [..., D] int8, ``scales`` [..., ceil(D / 128)] fp32; a value is code * scale.

    ``dtype``: that of the tensor it was made from (calls that pack set it, also of one given to write to), which a backward call goes by
    where no tensor of its arguments says what type its gradients have; None where it was put together without."""
    dtype = None

    def __new__(cls, codes, scales, dtype=None):
        if dtype is not None and dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {dtype}")
        self = super().__new__(cls, codes, scales)
        self.dtype = dtype
        return self

    def _replace(self, **fields):
        return Packed(fields.pop("codes", self.codes), fields.pop("scales", self.scales), fields.pop("dtype", self.dtype), **fields)

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device

    def dim(self) -> int:
        return self.codes.dim()


def _scale_shape(shape):
    return (*shape[:-1], (shape[-1] + ACT_GROUP - 1) // ACT_GROUP)


def _good(t, device, dtype, shape) -> bool:
    """Whether t is a dense tensor of this kind: a small call's time is mostly the host's, so the good case is one line."""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()


def _new_packed(shape, device, dtype):
    return Packed(torch.empty(shape, dtype=torch.int8, device=device),
                  torch.empty(_scale_shape(shape), dtype=torch.float32, device=device), dtype)


def _check_packed(p, name, shape, device):
    if _good(p.codes, device, torch.int8, shape) and _good(p.scales, device, torch.float32, _scale_shape(shape)) and device.type == "cuda":
        return
    _required(device, torch.int8, **{f"{name}.codes": p.codes})
    _required(device, torch.float32, **{f"{name}.scales": p.scales})
    if tuple(p.codes.shape) != tuple(shape) or tuple(p.scales.shape) != _scale_shape(shape):
        raise ValueError(f"{name} must be codes {tuple(shape)} and scales {_scale_shape(shape)}, got {tuple(p.codes.shape)} "
                         f"and {tuple(p.scales.shape)}")


def _packed_out(pack, name, shape, device, dtype):
    """A forward's 8-bit copy of a tensor of dtype: allocated for True, checked when given, None for False."""
    if pack is None or pack is False:
        return None
    if pack is True:
        return _new_packed(shape, device, dtype)
    if not isinstance(pack, Packed):
        raise ValueError(f"{name} must be a Packed")
    _check_packed(pack, name, shape, device)
    pack.dtype = dtype
    return pack


def _row_stride(t, name):
    """Elements from one row (last axis) to the next: the leading axes have to be evenly spaced."""
    if t.is_contiguous():
        return t.shape[-1]
    size, stride = t.shape, t.stride()
    if size[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the last axis must be dense")
    row, span = None, 0
    for n, s in zip(reversed(size[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if row is None:
            row, span = s, s * n
        elif s != span:
            raise ValueError(f"{name}: rows must be evenly spaced, got strides {tuple(stride)}")
        else:
            span = s * n
    if row is None:
        return size[-1]
    if row < size[-1]:
        raise ValueError(f"{name}: rows must not overlap, got strides {tuple(stride)}")
    return row


def _rows(t, name, device, dtype, shape):
    """Checks a tensor of rows of any stride; returns (address, stride)."""
    if _good(t, device, dtype, shape) and device.type == "cuda":
        return t.data_ptr(), shape[-1]
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call is on {device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr(), _row_stride(t, name)


def _saved(t, name, device, dtype, shape):
    """Checks a saved activation, elements of any row stride or a Packed; returns (address, stride, scales)."""
    if isinstance(t, Packed):
        _check_packed(t, name, shape, device)
        return t.codes.data_ptr(), shape[-1], t.scales.data_ptr()
    return (*_rows(t, name, device, dtype, shape), None)


def _two(t):
    """(R, D) of [..., D]."""
    return t.numel() // max(t.shape[-1], 1) if t.dim() else 0, t.shape[-1] if t.dim() else 0


@_on_stream
def act_pack(x, *, out=None):
    """x [..., D] (bf16 or fp32, rows of any even spacing) in 8 bits (``kda_act_pack``).  Returns a :class:`Packed`; ``out``: one
    to write to."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be a device tensor [..., D] with D >= 1")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    at, stride = _rows(x, "x", x.device, x.dtype, x.shape)
    R, D = _two(x)
    out = _packed_out(True if out is None else out, "out", x.shape, x.device, x.dtype)
    _call("kda_act_pack", (_DTYPES[x.dtype], at, stride, R, D, out.codes.data_ptr(), out.scales.data_ptr()), x.device)
    return out


@_on_stream
def act_unpack(packed, *, dtype=torch.bfloat16, out=None):
    """The values of a :class:`Packed` as a dense tensor of ``dtype`` (``kda_act_unpack``), or in ``out``."""
    if not isinstance(packed, Packed) or not isinstance(packed.codes, torch.Tensor) or packed.codes.dim() < 1:
        raise ValueError("packed must be a Packed")
    dev, shape = packed.codes.device, packed.codes.shape
    if shape[-1] < 1:
        raise ValueError("packed must be [..., D] with D >= 1")
    _check_packed(packed, "packed", shape, dev)
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {dtype}")
        out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        if out.dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {out.dtype}")
        _check_tensors(dev, out.dtype, out=out)
        if out.shape != shape:
            raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    R, D = _two(packed.codes)
    _call("kda_act_unpack", (_DTYPES[out.dtype], packed.codes.data_ptr(), packed.scales.data_ptr(), R, D, out.data_ptr()), dev)
    return out
