"""What stands between two blocks of a model (``kda_block_norm_*``): the norm after a block's output, its gate, the residual
stream, and the norm before the next block, in one pass over the rows.

    u  = post_weight * y / rms(y)
    x' = x + scale * res_scale * Sigmoid(gate) * u
    n  = pre_weight * x' / rms(x')

Every call also takes ``stream`` (a torch.cuda.Stream; None: the current one), on which it runs and allocates.  Outputs
carry no autograd history: a training step calls :func:`block_norm_bwd` itself.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _DTYPES, BlockNormBwdArgs, BlockNormFwdArgs, _dev
from .act import Packed, _good, _packed_out, _rows, _saved, _two
from .linear import _at, _call, _check_tensors, _like, _need, _on_stream, _required, _workspace


class BlockNormGrads(NamedTuple):
    dx: torch.Tensor
    dy: torch.Tensor | None
    dgate: torch.Tensor | None
    dpost_weight: torch.Tensor | None
    dres_scale: torch.Tensor | None
    dpre_weight: torch.Tensor | None


class BlockNormSaved(NamedTuple):
    """What the backward pass reads, in 8 bits; in the order of its arguments."""
    x_new: Packed
    y: Packed | None
    gate: Packed | None


def _weights(device, shape, post_weight, res_scale, pre_weight):
    """Checks the weights, each [D]; returns their addresses."""
    shape = shape[-1:]
    for name, w in (("post_weight", post_weight), ("res_scale", res_scale), ("pre_weight", pre_weight)):
        if w is not None and not _good(w, device, torch.float32, shape):
            _check_tensors(device, torch.float32, **{name: w})
            if w.shape != shape:
                raise ValueError(f"{name} must be [D] = {list(shape)}, got {tuple(w.shape)}")
    return _at(post_weight), _at(res_scale), _at(pre_weight)


def _stream_rows(x, name):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError(f"{name} must be a device tensor [..., D]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if not x.is_cuda or not x.is_contiguous():
        _dev(x, name)


@_on_stream
def block_norm_fwd(x, y=None, *, gate=None, post_weight=None, res_scale=None, scale: float = 1.0, pre_weight=None,
                   eps: float = 1e-6, x_out=None, n_out=None, pack=False):
    """Forward (``kda_block_norm_fwd``).

    x: the residual stream [..., D] (the blocks' dtype, or fp32 next to bf16 blocks); y, gate: the block's output and its gate's
    logits, like x in the blocks' dtype, rows of any even spacing; post_weight, res_scale, pre_weight: [D] fp32, each optional
    (without pre_weight there is no n).  Without y there is no block before: x' is x itself and only n is computed (in
    ``n_out``'s dtype when given, else x's).  x_out may be x.  ``pack`` (True or a :class:`BlockNormSaved` to write to): x', y
    and the gate in 8 bits as well.  Returns (x', n or None), with ``pack`` (x', n or None, BlockNormSaved)."""
    if n_out is not None and pre_weight is None:
        raise ValueError("n_out without pre_weight: there is no n")
    if pack is not None and not isinstance(pack, (bool, BlockNormSaved)):
        raise ValueError("pack must be True, False or a BlockNormSaved")
    _stream_rows(x, "x")
    dev, shape = x.device, x.shape
    R, D = _two(x)
    if y is not None:
        dtype = y.dtype if isinstance(y, torch.Tensor) else None
    else:
        dtype = x.dtype if n_out is None else n_out.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    y_at = x_out_at = gate_at = None
    y_stride = gate_stride = D
    if y is not None:
        y_at, y_stride = _rows(y, "y", dev, dtype, shape)
        x_out = _like(x_out, "x_out", x)
        x_out_at = x_out.data_ptr()
    elif x_out is not None:
        raise ValueError("x_out without y: there is no new residual stream")
    else:
        x_out = x
    if gate is not None:
        gate_at, gate_stride = _rows(gate, "gate", dev, dtype, shape)
    weights = _weights(dev, shape, post_weight, res_scale, pre_weight)
    n = None
    if pre_weight is not None:
        if n_out is None:
            n = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _check_tensors(dev, dtype, n_out=n_out)
            if n_out.shape != shape:
                raise ValueError(f"n_out must be {tuple(shape)}, got {tuple(n_out.shape)}")
            n = n_out
    a = BlockNormFwdArgs(R, D, _DTYPES[dtype], _DTYPES[x.dtype], x.data_ptr(), y_at, y_stride, gate_at, gate_stride, *weights,
                         scale, eps, x_out_at, _at(n))
    saved = None
    if pack is not None and pack is not False:
        given = pack if isinstance(pack, BlockNormSaved) else (True, y is not None, gate is not None)
        if (given[1] is None and y is not None) or (given[2] is None and gate is not None):
            raise ValueError("pack must hold a Packed for each of x_new, y and gate that there is")
        saved = BlockNormSaved(_packed_out(given[0], "pack.x_new", shape, dev, x.dtype),
                               _packed_out(given[1] if y is not None else None, "pack.y", shape, dev, dtype),
                               _packed_out(given[2] if gate is not None else None, "pack.gate", shape, dev, dtype))
        for name, p in zip(("x", "y", "gate"), saved):
            if p is not None:
                setattr(a, name + "_codes", p.codes.data_ptr())
                setattr(a, name + "_scales", p.scales.data_ptr())
    _call("kda_block_norm_fwd", (ctypes.byref(a),), dev)
    return (x_out, n, saved) if saved is not None else (x_out, n)


def _types(x_new, y, gate, dx_new, dn, dtype, dx, dy, dgate):
    """(the blocks' dtype, the residual stream's) as the arguments name them: tensors first, since a call checks them, then what a
    Packed says it was made from, then what the one type settles of the other."""
    def named(*args):
        for kind in (torch.Tensor, Packed):
            for t in args:
                if isinstance(t, kind) and t.dtype is not None:
                    return t.dtype
        return None
    x_dtype = dx_new.dtype if isinstance(dx_new, torch.Tensor) else named(x_new, dx)
    if dtype is None:
        dtype = dn.dtype if isinstance(dn, torch.Tensor) else named(y, gate, dy, dgate)
    if dtype is None and (x_dtype is torch.bfloat16 or (y is None and dn is None)):
        dtype = x_dtype                        # a bf16 stream has bf16 blocks; without blocks no value is of their type
    if x_dtype is None and dtype is torch.float32:
        x_dtype = dtype                        # fp32 blocks have an fp32 stream
    if dtype is None:
        raise ValueError("nothing names the blocks' dtype: give dtype, or y or the gate as a Packed with its dtype")
    if x_dtype is None:
        raise ValueError("nothing names the residual stream's dtype: give dx, or x_new as a Packed with its dtype")
    if dtype not in _DTYPES or x_dtype not in _DTYPES:
        raise ValueError(f"unsupported dtypes {dtype}, {x_dtype}")
    return dtype, x_dtype


@_on_stream
def block_norm_bwd(x_new, y, dx_new, dn=None, *, gate=None, post_weight=None, res_scale=None, scale: float = 1.0,
                   pre_weight=None, eps: float = 1e-6, need_dweights: bool = True, dtype=None, dx=None, dy=None, dgate=None,
                   workspace=None) -> BlockNormGrads:
    """Gradients of :func:`block_norm_fwd` (``kda_block_norm_bwd``), given ``dx_new`` (gradient of x', x's dtype) and ``dn``
    (gradient of n, the blocks' dtype), one of which may be None (zeros).

    x_new: x' as the forward returned it (read, and required, with ``dn`` only); y, gate: its inputs; each a tensor or a
    :class:`Packed`.  ``dtype``: the blocks' dtype (None: that of dn, y, the gate, dy or dgate; the stream's is that of dx_new,
    x_new or dx).  A type that none of these names (a Packed may not know its own) is not guessed: the call is refused.  dx may be dx_new;
    dy and dgate may go to rows of any even spacing.  Returns a :class:`BlockNormGrads`, dx in the stream's dtype, dy and dgate in the
    blocks'; the weights' gradients are fp32, None where there is no weight or without ``need_dweights``."""
    if dy is not None and y is None:
        raise ValueError("dy without y: there is no such gradient")
    if dgate is not None and gate is None:
        raise ValueError("dgate without gate: there is no such gradient")
    ref = dx_new if dx_new is not None else dn
    _stream_rows(ref, "dx_new" if dx_new is not None else "dn")
    dev, shape = ref.device, ref.shape
    R, D = _two(ref)
    if dn is not None:
        _stream_rows(dn, "dn")
    dtype, x_dtype = _types(x_new, y, gate, dx_new, dn, dtype, dx, dy, dgate)
    if y is None and (gate is not None or post_weight is not None or res_scale is not None):
        raise ValueError("gate, post_weight and res_scale belong to y, which is None")
    if dn is not None and pre_weight is None:
        raise ValueError("dn without pre_weight")
    x_at = x_scales = y_at = y_scales = gate_at = gate_scales = dy_at = dgate_at = None
    y_stride = gate_stride = dy_stride = dgate_stride = D
    if dn is not None:
        _check_tensors(dev, dtype, dn=dn)
        if dn.shape != shape:
            raise ValueError(f"dn must be {tuple(shape)}, got {tuple(dn.shape)}")
        if isinstance(x_new, Packed):
            x_at, _, x_scales = _saved(x_new, "x_new", dev, x_dtype, shape)
        else:
            if not _good(x_new, dev, x_dtype, shape):
                _required(dev, x_dtype, x_new=x_new)
                if x_new.shape != shape:
                    raise ValueError(f"x_new must be {tuple(shape)}, got {tuple(x_new.shape)}")
            x_at = x_new.data_ptr()
    if dx is None:
        dx = torch.empty(shape, dtype=x_dtype, device=dev)
    else:
        _check_tensors(dev, x_dtype, dx=dx)
        if dx.shape != shape:
            raise ValueError(f"dx must be {tuple(shape)}, got {tuple(dx.shape)}")
    if y is not None:
        y_at, y_stride, y_scales = _saved(y, "y", dev, dtype, shape)
        if dy is None:
            dy = torch.empty(shape, dtype=dtype, device=dev)
            dy_at = dy.data_ptr()
        else:
            dy_at, dy_stride = _rows(dy, "dy", dev, dtype, shape)
    if gate is not None:
        gate_at, gate_stride, gate_scales = _saved(gate, "gate", dev, dtype, shape)
        if dgate is None:
            dgate = torch.empty(shape, dtype=dtype, device=dev)
            dgate_at = dgate.data_ptr()
        else:
            dgate_at, dgate_stride = _rows(dgate, "dgate", dev, dtype, shape)
    weights = _weights(dev, shape, post_weight, res_scale, pre_weight)
    grads = [torch.empty_like(w) if w is not None and need_dweights else None for w in (post_weight, res_scale, pre_weight)]
    a = BlockNormBwdArgs(R, D, _DTYPES[dtype], _DTYPES[x_dtype], x_at, x_scales, y_at, y_stride, y_scales, gate_at, gate_stride,
                         gate_scales, *weights, scale, eps, _at(dx_new), _at(dn), dx.data_ptr(), dy_at, dy_stride, dgate_at,
                         dgate_stride, *map(_at, grads))
    workspace = _workspace("kda_block_norm_bwd_workspace_size", a, workspace, dev)
    _call("kda_block_norm_bwd", (ctypes.byref(a),), dev)
    return BlockNormGrads(dx, dy, dgate, *grads)


def block_norm_bwd_workspace_size(x_new, *, weights: int = 3) -> int:
    """Workspace bytes :func:`block_norm_bwd` needs for x_new [..., D] (where the call has none: dx_new) when gradients of ``weights``
    weights are wanted."""
    if not isinstance(x_new, (torch.Tensor, Packed)):
        raise ValueError("x_new must be a tensor or a Packed; without one give dx_new")
    R, D = _two(x_new.codes if isinstance(x_new, Packed) else x_new)
    x_dtype = x_new.dtype
    if x_dtype is not None and x_dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x_dtype}")
    need = 0
    # the stream does not say what blocks it has, but for a bf16 one
    for dtype in (torch.bfloat16,) if x_dtype is torch.bfloat16 else (torch.bfloat16, torch.float32):
        a = BlockNormBwdArgs(R, D, _DTYPES[dtype], _DTYPES[dtype], scale=1.0)
        a.d_pre_weight = 16 if weights else None   # only whether one is given is read
        need = max(need, _need("kda_block_norm_bwd_workspace_size", a))
    return need
