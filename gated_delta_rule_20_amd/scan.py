"""The gated scan (``kda_gated_scan_*``): per channel h_t = a_t h_{t-1} + m_t x_t.

a_t = exp(g_t) with log-decays g, or with ``A_log`` ([C] fp32) and logits g the gate of eq. (5),
g_t = g_min * Sigmoid(exp(A_log) * logit); m_t is 1, or 1 - a_t with ``complement``.

Every call also takes ``stream`` (a torch.cuda.Stream; None: the current one), on which it runs and allocates.  Outputs
carry no autograd history: a training step calls :func:`gated_scan_bwd` itself.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DTYPES, GatedScanBwdArgs, GatedScanFwdArgs, GatedScanStepArgs
from .act import Packed, _good, _packed_out, _rows, _saved
from .linear import _at, _call, _check_tensors, _like, _need, _on_stream, _required, _workspace


def _decay(g, name, dtype, shape, A_log, device):
    """Checks g (of dtype or fp32) and A_log; returns (address, stride, kda_dtype_t)."""
    if not isinstance(g, torch.Tensor):
        raise ValueError(f"{name} must be a device tensor")
    if g.dtype is not dtype and g.dtype is not torch.float32:
        raise ValueError(f"{name} must be {dtype} or torch.float32, got {g.dtype}")
    if A_log is not None and not _good(A_log, device, torch.float32, shape[-1:]):
        _check_tensors(device, torch.float32, A_log=A_log)
        if A_log.shape != (shape[-1],):
            raise ValueError(f"A_log must be [C] = [{shape[-1]}], got {tuple(A_log.shape)}")
    return (*_rows(g, name, device, g.dtype, shape), _DTYPES[g.dtype])


def _tokens(t, name, cu_seqlens):
    """(B, T, C, N) of t [B, T, C], or with cu_seqlens of [T, C] (a leading 1 allowed)."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if cu_seqlens is None:
        if t.dim() != 3:
            raise ValueError(f"{name} must be [B, T, C], got {tuple(t.shape)}")
        return t.shape[0], t.shape[1], t.shape[2], t.shape[0]
    _check_tensors(t.device, torch.int32, cu_seqlens=cu_seqlens)
    if t.dim() not in (2, 3) or (t.dim() == 3 and t.shape[0] != 1):
        raise ValueError(f"with cu_seqlens {name} must be [T, C], got {tuple(t.shape)}")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError(f"cu_seqlens must be [N + 1] with N >= 1, got {tuple(cu_seqlens.shape)}")
    return 1, t.shape[-2], t.shape[-1], cu_seqlens.shape[0] - 1


def _state(t, name, shape, device):
    if t is not None and not _good(t, device, torch.float32, shape):
        _check_tensors(device, torch.float32, **{name: t})
        if t.shape != shape:
            raise ValueError(f"{name} must be [N, C] = {shape}, got {tuple(t.shape)}")


def _strided_out(t, name, ref):
    """A result shaped like ref, dense unless a tensor of rows is given; returns (tensor, address, stride)."""
    if t is None:
        t = torch.empty(ref.shape, dtype=ref.dtype, device=ref.device)
        return t, t.data_ptr(), ref.shape[-1]
    return (t, *_rows(t, name, ref.device, ref.dtype, ref.shape))


@_on_stream
def gated_scan_fwd(x, g, *, A_log=None, g_min: float = -5.0, complement: bool = False, cu_seqlens=None, initial_state=None,
                   output_final_state: bool = True, out=None, final_state=None, pack=False, workspace=None):
    """Forward over whole sequences (``kda_gated_scan_fwd``).

    x, g: [B, T, C] (bf16 or fp32; g also fp32 next to bf16 x), rows of any even spacing (halves of one projection, say); with
    cu_seqlens ([N+1] int32 on the device) packed: [T, C].  initial_state / final_state: [N, C] fp32 (may be one tensor).
    ``pack``: True (or a :class:`Packed` to write to): h in 8 bits as well, for :func:`gated_scan_bwd`.
    Returns (h, final_state or None), with ``pack`` (h, final_state or None, Packed)."""
    B, T, C, N = _tokens(x, "x", cu_seqlens)
    dev, shape = x.device, (N, C)
    x_at, x_stride = _rows(x, "x", dev, x.dtype, x.shape)
    g_at, g_stride, g_dtype = _decay(g, "g", x.dtype, x.shape, A_log, dev)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _like(out, "out", x)
    _state(initial_state, "initial_state", shape, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty(shape, dtype=torch.float32, device=dev)
    _state(final_state, "final_state", shape, dev)
    h8 = _packed_out(pack, "pack", x.shape, dev, x.dtype)
    a = GatedScanFwdArgs(B, T, C, _DTYPES[x.dtype], g_dtype, x_at, x_stride, g_at, g_stride, _at(A_log), g_min, complement,
                         _at(cu_seqlens), N, _at(initial_state), _at(out), _at(final_state),
                         _at(h8.codes) if h8 else None, _at(h8.scales) if h8 else None, None, 0)
    workspace = _workspace("kda_gated_scan_fwd_workspace_size", a, workspace, dev)
    _call("kda_gated_scan_fwd", (ctypes.byref(a),), dev)
    return (out, final_state, h8) if h8 else (out, final_state)


@_on_stream
def gated_scan_bwd(x, g, h, d_h, *, A_log=None, g_min: float = -5.0, complement: bool = False, cu_seqlens=None,
                   initial_state=None, dfinal_state=None, need_dg: bool = True, dx=None, dg=None, dA_log=None,
                   dinitial_state=None, workspace=None):
    """Gradients of :func:`gated_scan_fwd` for the same arguments (``kda_gated_scan_bwd``), given ``d_h`` (like h) and
    ``dfinal_state`` ([N, C] fp32, None: zeros).

    h: what the forward returned, or its :class:`Packed`; read (and required) with ``need_dg`` only.  x: read with ``complement``
    and ``need_dg`` only (None otherwise), a tensor or a Packed.  dx, dg: results may go to rows of any even spacing.  A log-decay above 0,
    which the forward counts as 0, gets the gradient at 0 (not the 0 of a clamped value); an infinite logit has none.
    Returns (dx, dg, dA_log, dinitial_state); dg, of g's dtype, is None without ``need_dg``, dA_log fp32 None without A_log or
    ``need_dg``."""
    B, T, C, N = _tokens(d_h, "d_h", cu_seqlens)
    dev, dtype, rows, shape = d_h.device, d_h.dtype, d_h.shape, (N, C)
    if not d_h.is_contiguous():
        _required(dev, dtype, d_h=d_h)
    g_at, g_stride, g_dtype = _decay(g, "g", dtype, rows, A_log, dev)
    x_at, x_stride, x_scales = None, C, None
    h_at, h_scales = None, None
    if need_dg:
        if isinstance(h, Packed):
            h_at, _, h_scales = _saved(h, "h", dev, dtype, rows)
        else:
            if not _good(h, dev, dtype, rows):
                _required(dev, dtype, h=h)
                if h.shape != rows:
                    raise ValueError(f"h must have d_h's shape {tuple(rows)}, got {tuple(h.shape)}")
            h_at = h.data_ptr()
        if complement:
            x_at, x_stride, x_scales = _saved(x, "x", dev, dtype, rows)
    _state(initial_state, "initial_state", shape, dev)
    _state(dfinal_state, "dfinal_state", shape, dev)
    dx, dx_at, dx_stride = _strided_out(dx, "dx", d_h)
    dg_at, dg_stride = None, C
    if need_dg:
        dg, dg_at, dg_stride = _strided_out(dg, "dg", g)
    else:
        dg = None
    if A_log is not None and need_dg:
        dA_log = _like(dA_log, "dA_log", A_log)
    else:
        dA_log = None
    if dinitial_state is None:
        dinitial_state = torch.empty(shape, dtype=torch.float32, device=dev)
    _state(dinitial_state, "dinitial_state", shape, dev)
    a = GatedScanBwdArgs(B, T, C, _DTYPES[dtype], g_dtype, x_at, x_stride, x_scales, g_at, g_stride, _at(A_log), g_min,
                         complement, _at(cu_seqlens), N, _at(initial_state), h_at, h_scales, _at(d_h), _at(dfinal_state),
                         dx_at, dx_stride, dg_at, dg_stride, _at(dA_log), _at(dinitial_state), None, 0)
    workspace = _workspace("kda_gated_scan_bwd_workspace_size", a, workspace, dev)
    _call("kda_gated_scan_bwd", (ctypes.byref(a),), dev)
    return dx, dg, dA_log, dinitial_state


@_on_stream
def gated_scan_step(x, g, state, *, A_log=None, g_min: float = -5.0, complement: bool = False, slots=None, new_state=None,
                    out=None):
    """One token for each of N sequences (``kda_gated_scan_step``).

    x, g: [N, C]; state: [n_slots, C] fp32, updated in place unless ``new_state`` (same shape) receives the results.  slots:
    [N] int32, the slot of each sequence's state (None: slot n); rows whose slot is out of range, or that an earlier row
    already names, are empty places: their output is zero and no state changes.  Returns h [N, C]."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a device tensor [N, C]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    dev, (N, C) = x.device, x.shape
    x_at, x_stride = _rows(x, "x", dev, x.dtype, x.shape)
    g_at, g_stride, g_dtype = _decay(g, "g", x.dtype, x.shape, A_log, dev)
    _required(dev, torch.float32, state=state)
    _check_tensors(dev, torch.float32, new_state=new_state)
    if state.dim() != 2 or state.shape[1] != C:
        raise ValueError(f"state must be [n_slots, C] with C = {C}, got {tuple(state.shape)}")
    if slots is not None:
        _check_tensors(dev, torch.int32, slots=slots)
        if slots.dim() != 1 or slots.shape[0] != N:
            raise ValueError(f"slots must be [N] = [{N}], got {tuple(slots.shape)}")
    if new_state is None:
        new_state = state
    elif new_state.shape != state.shape:
        raise ValueError(f"new_state must have state's shape {tuple(state.shape)}, got {tuple(new_state.shape)}")
    if out is None:
        out = torch.empty((N, C), dtype=x.dtype, device=dev)
    else:
        _like(out, "out", x)
    a = GatedScanStepArgs(N, C, _DTYPES[x.dtype], g_dtype, x_at, x_stride, g_at, g_stride, _at(A_log), g_min, complement,
                          _at(slots), state.shape[0], state.data_ptr(), new_state.data_ptr(), out.data_ptr())
    _call("kda_gated_scan_step", (ctypes.byref(a),), dev)
    return out


def gated_scan_fwd_workspace_size(x, *, g_dtype=None, cu_seqlens=None, same_states: bool = False) -> int:
    """Workspace bytes :func:`gated_scan_fwd` needs for x [B, T, C] (or [T, C] with cu_seqlens) and g of ``g_dtype`` (None: x's);
    ``same_states``: initial_state is final_state."""
    B, T, C, N = _tokens(x, "x", cu_seqlens)
    a = GatedScanFwdArgs(B, T, C, _DTYPES[x.dtype], _DTYPES[g_dtype or x.dtype], cu_seqlens=_at(cu_seqlens), N=N)
    if same_states:                            # only whether they overlap is read
        a.initial_state = a.final_state = 16
    return _need("kda_gated_scan_fwd_workspace_size", a)


def gated_scan_bwd_workspace_size(d_h, *, g_dtype=None, cu_seqlens=None, A_log: bool = False, same_states: bool = False) -> int:
    """Workspace bytes :func:`gated_scan_bwd` needs for d_h [B, T, C] (or [T, C] with cu_seqlens); ``A_log``: its gradient is wanted;
    ``same_states``: dinitial_state is dfinal_state."""
    B, T, C, N = _tokens(d_h, "d_h", cu_seqlens)
    a = GatedScanBwdArgs(B, T, C, _DTYPES[d_h.dtype], _DTYPES[g_dtype or d_h.dtype], cu_seqlens=_at(cu_seqlens), N=N)
    a.dA_log = 16 if A_log else None           # only whether it is given is read
    if same_states:
        a.d_initial_state = a.d_final_state = 16
    return _need("kda_gated_scan_bwd_workspace_size", a)
