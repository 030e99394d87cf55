"""Linear attention with a decay for each head (``kda_linear_*``).

The recurrence next to KDA's that writes without the delta rule and forgets with
one scalar per head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DTYPES, LinearBwdArgs, LinearFwdArgs, LinearStepArgs, _check, _dev, _ptr, _stream, load_library


def _on_device(device, **tensors):
    """Every given tensor lives on ``device``."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the call is on {device}")


def _call(fn, args, stream, device):
    """The library launches on the current device: make it the tensors' own."""
    lib = load_library()
    if device.index == torch.cuda.current_device():
        status = getattr(lib, fn)(*args, _stream(stream, device))
    else:
        with torch.cuda.device(device):
            status = getattr(lib, fn)(*args, _stream(stream, device))
    _check(lib, fn, status)


def _heads(q, k, v, g):
    """Checks q, k [..., Hk, Dk], v [..., H, Dv] and g [..., H] or [H]; returns (H, Hk, Dk, Dv, g_per_head)."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    _dev(g, "g", torch.float32)
    _on_device(q.device, k=k, v=v, g=g)
    if k.shape != q.shape:
        raise ValueError(f"k must have q's shape {tuple(q.shape)}, got {tuple(k.shape)}")
    if v.dim() != q.dim() or v.shape[:-2] != q.shape[:-2]:
        raise ValueError(f"v must be [..., H, Dv] over q's leading axes {tuple(q.shape[:-2])}, got {tuple(v.shape)}")
    H, Hk = v.shape[-2], q.shape[-2]
    if Hk < 1 or H % Hk != 0:
        raise ValueError(f"v's {H} heads must be a multiple of q's {Hk}")
    per_head = g.dim() == 1
    if not (tuple(g.shape) == (H,) if per_head else g.shape == v.shape[:-1]):
        raise ValueError(f"g must be [H] = [{H}] or {tuple(v.shape[:-1])}, got {tuple(g.shape)}")
    return H, Hk, q.shape[-1], v.shape[-1], per_head


def _sequences(q, v, cu_seqlens):
    """(B, T, N) of q [B, T, Hk, Dk], or with cu_seqlens of [T, Hk, Dk] (a leading 1 allowed)."""
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError(f"q must be [B, T, Hk, Dk], got {tuple(q.shape)}")
        return q.shape[0], q.shape[1], q.shape[0]
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    _on_device(q.device, cu_seqlens=cu_seqlens)
    if q.dim() not in (3, 4) or (q.dim() == 4 and q.shape[0] != 1):
        raise ValueError(f"with cu_seqlens q must be [T, Hk, Dk], got {tuple(q.shape)}")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError(f"cu_seqlens must be [N + 1] with N >= 1, got {tuple(cu_seqlens.shape)}")
    return 1, q.shape[-3], cu_seqlens.shape[0] - 1


def _state(t, name, shape, device):
    if t is not None:
        _dev(t, name, torch.float32)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be [N, H, Dk, Dv] = {shape}, got {tuple(t.shape)}")
        _on_device(device, **{name: t})
    return t


def _like(t, name, ref, dtype=None):
    """An output: allocated like ref when not given, checked when given."""
    if t is None:
        return torch.empty(ref.shape, dtype=dtype or ref.dtype, device=ref.device)
    _dev(t, name, dtype or ref.dtype)
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have shape {tuple(ref.shape)}, got {tuple(t.shape)}")
    _on_device(ref.device, **{name: t})
    return t


def _workspace(fn, a, workspace, device):
    """Sets the workspace the call needs (allocated when not given); returns it so that it outlives the call."""
    need = _need(fn, a)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is not None:
        _dev(workspace, "workspace")
        _on_device(device, workspace=workspace)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return workspace


def linear_chunk_fwd(q, k, v, g, *, scale: float = 1.0, cu_seqlens=None, initial_state=None,
                     output_final_state: bool = True, out=None, final_state=None, workspace=None, stream=None,
                     checkpoints=None, checkpoint_every: int = 0):
    """Forward over whole sequences (``kda_linear_chunk_fwd``).

    q, k: [B, T, Hk, Dk]; v: [B, T, H, Dv] (bf16 or fp32; H a multiple of Hk: value head h reads query / key head
    h // (H // Hk)); g: log-decays [B, T, H] or [H] fp32.  With cu_seqlens ([N+1] int32 on the device) the token axis is
    packed: [T, H, D].  initial_state / final_state: [N, H, Dk, Dv] fp32 (may be one tensor).  checkpoints /
    checkpoint_every as for :func:`chunk_fwd`.  Returns (o, final_state or None)."""
    H, Hk, Dk, Dv, per_head = _heads(q, k, v, g)
    B, T, N = _sequences(q, v, cu_seqlens)
    dev, shape = q.device, (N, H, Dk, Dv)
    out = _like(out, "out", v)
    _state(initial_state, "initial_state", shape, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty(shape, dtype=torch.float32, device=dev)
    _state(final_state, "final_state", shape, dev)
    slots = 0
    if checkpoints is not None:
        _dev(checkpoints, "checkpoints", torch.float32)
        _on_device(dev, checkpoints=checkpoints)
        if (checkpoints.dim() != 5 or checkpoints.shape[0] != N or checkpoints.shape[1] < 1
                or tuple(checkpoints.shape[2:]) != shape[1:] or checkpoint_every < 1):
            raise ValueError(f"checkpoints must be [N, slots >= 1, H, Dk, Dv] with N, H, Dk, Dv = {shape} and "
                             f"checkpoint_every >= 1; got {tuple(checkpoints.shape)}, every={checkpoint_every}")
        slots = checkpoints.shape[1]
    a = LinearFwdArgs(B, T, H, Hk, Dk, Dv, _DTYPES[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(g), per_head, scale,
                      _ptr(cu_seqlens), N, _ptr(initial_state), _ptr(out), _ptr(final_state), None, 0,
                      _ptr(checkpoints), checkpoint_every if slots else 0, slots)
    workspace = _workspace("kda_linear_chunk_fwd_workspace_size", a, workspace, dev)
    _call("kda_linear_chunk_fwd", (ctypes.byref(a),), stream, dev)
    return out, final_state


def linear_chunk_bwd(q, k, v, g, d_o, *, scale: float = 1.0, cu_seqlens=None, initial_state=None, dfinal_state=None,
                     need_dg: bool = True, dq=None, dk=None, dv=None, dg=None, dinitial_state=None, workspace=None,
                     stream=None):
    """Gradients of :func:`linear_chunk_fwd` (``kda_linear_chunk_bwd``) for the same arguments, given ``d_o`` (shaped
    like o, in its dtype) and ``dfinal_state`` ([N, H, Dk, Dv] fp32, None: zeros).  Returns (dq, dk, dv, dg, dinitial_state):
    the first three shaped and typed like q, k, v; dg fp32 shaped like g (None without ``need_dg``)."""
    H, Hk, Dk, Dv, per_head = _heads(q, k, v, g)
    B, T, N = _sequences(q, v, cu_seqlens)
    dev, shape = q.device, (N, H, Dk, Dv)
    _dev(d_o, "d_o", q.dtype)
    if d_o.shape != v.shape:
        raise ValueError(f"d_o must have v's shape {tuple(v.shape)}, got {tuple(d_o.shape)}")
    _on_device(dev, d_o=d_o)
    _state(initial_state, "initial_state", shape, dev)
    _state(dfinal_state, "dfinal_state", shape, dev)
    dq, dk, dv = _like(dq, "dq", q), _like(dk, "dk", k), _like(dv, "dv", v)
    dg = _like(dg, "dg", g) if need_dg else None
    if dinitial_state is None:
        dinitial_state = torch.empty(shape, dtype=torch.float32, device=dev)
    _state(dinitial_state, "dinitial_state", shape, dev)
    a = LinearBwdArgs(B, T, H, Hk, Dk, Dv, _DTYPES[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(g), per_head, scale,
                      _ptr(cu_seqlens), N, _ptr(initial_state), _ptr(d_o), _ptr(dfinal_state), _ptr(dq), _ptr(dk),
                      _ptr(dv), _ptr(dg), _ptr(dinitial_state), None, 0)
    workspace = _workspace("kda_linear_chunk_bwd_workspace_size", a, workspace, dev)
    _call("kda_linear_chunk_bwd", (ctypes.byref(a),), stream, dev)
    return dq, dk, dv, dg, dinitial_state


def linear_chunk_fwd_workspace_size(q, v, *, cu_seqlens=None) -> int:
    """Workspace bytes :func:`linear_chunk_fwd` needs for q [B, T, Hk, Dk] (or [T, Hk, Dk] with cu_seqlens) and v."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, T, N = _sequences(q, v, cu_seqlens)
    a = LinearFwdArgs(B, T, v.shape[-2], q.shape[-2], q.shape[-1], v.shape[-1], _DTYPES[q.dtype], scale=1.0,
                      cu_seqlens=_ptr(cu_seqlens), N=N)
    return _need("kda_linear_chunk_fwd_workspace_size", a)


def linear_chunk_bwd_workspace_size(q, v, *, cu_seqlens=None, g_per_head: bool = False, need_dg: bool = True,
                                    dfinal_state: bool = False) -> int:
    """Workspace bytes :func:`linear_chunk_bwd` needs; the flags say whether g is [H], whether dg is wanted and whether
    dfinal_state is given."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, T, N = _sequences(q, v, cu_seqlens)
    a = LinearBwdArgs(B, T, v.shape[-2], q.shape[-2], q.shape[-1], v.shape[-1], _DTYPES[q.dtype], scale=1.0,
                      cu_seqlens=_ptr(cu_seqlens), N=N, g_per_head=g_per_head)
    a.dg = 16 if need_dg else None             # only whether they are given is read
    a.d_final_state = 16 if dfinal_state else None
    return _need("kda_linear_chunk_bwd_workspace_size", a)


def _need(fn, a) -> int:
    lib = load_library()
    need = ctypes.c_size_t(0)
    _check(lib, fn, getattr(lib, fn)(ctypes.byref(a), ctypes.byref(need)))
    return need.value


def linear_recurrent_step(q, k, v, g, state, *, scale: float = 1.0, slots=None, new_state=None, out=None, stream=None):
    """One token for each of N sequences (``kda_linear_recurrent_step``).

    q, k: [N, Hk, Dk]; v: [N, H, Dv] (bf16 or fp32; H a multiple of Hk); g: log-decays
    [N, H] or [H] fp32.  state: [n_slots, H, Dk, Dv] fp32, updated in place unless
    ``new_state`` (same shape) receives the results.  slots: [N] int32, the slot of
    each sequence's state (None: slot n); rows whose slot is out of range, or that an
    earlier row already names, are empty places: their output is zero and no state changes.
    Returns o [N, H, Dv]."""
    H, Hk, Dk, Dv, per_head = _heads(q, k, v, g)
    if q.dim() != 3:
        raise ValueError(f"q must be [N, Hk, Dk], got {tuple(q.shape)}")
    N = q.shape[0]
    _dev(state, "state", torch.float32)
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, Dk, Dv):
        raise ValueError(f"state must be [n_slots, H, Dk, Dv] with H, Dk, Dv = {(H, Dk, Dv)}, got {tuple(state.shape)}")
    if slots is not None:
        _dev(slots, "slots", torch.int32)
        if tuple(slots.shape) != (N,):
            raise ValueError(f"slots must be [N] = [{N}], got {tuple(slots.shape)}")
    if new_state is None:
        new_state = state
    elif _dev(new_state, "new_state", torch.float32).shape != state.shape:
        raise ValueError(f"new_state must have state's shape {tuple(state.shape)}, got {tuple(new_state.shape)}")
    if out is None:
        out = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    elif _dev(out, "out", q.dtype).shape != v.shape:
        raise ValueError(f"out must have v's shape {tuple(v.shape)}, got {tuple(out.shape)}")
    _on_device(q.device, state=state, slots=slots, new_state=new_state, out=out)
    a = LinearStepArgs(N, H, Hk, Dk, Dv, _DTYPES[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(g), per_head, scale,
                       _ptr(slots), state.shape[0], _ptr(state), _ptr(new_state), _ptr(out))
    _call("kda_linear_recurrent_step", (ctypes.byref(a),), stream, q.device)
    return out
