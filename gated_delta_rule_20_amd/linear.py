"""Linear attention with a decay for each head (``kda_linear_*``).

The recurrence next to KDA's that writes without the delta rule and forgets with
one scalar per head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t.

Every call also takes ``stream`` (a torch.cuda.Stream; None: the current one), on which
it runs and allocates.  Outputs carry no autograd history, whether or not the inputs require
gradients: a training step calls :func:`linear_chunk_bwd` itself, for instance from the
``backward`` of a ``torch.autograd.Function`` whose ``forward`` calls :func:`linear_chunk_fwd`.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _DTYPES, LinearBwdArgs, LinearFwdArgs, LinearStepArgs, _check, _dev, load_library


def _check_tensors(device, dtype, **tensors):
    """Every given tensor is contiguous, on ``device`` and of ``dtype`` (None: any).  A decode step's time is mostly the
    host's, so the good case is one line a tensor."""
    for name, t in tensors.items():
        if t is None or (isinstance(t, torch.Tensor) and t.device == device and (dtype is None or t.dtype is dtype)
                         and t.is_contiguous()):
            continue
        _dev(t, name, dtype)
        raise ValueError(f"{name} is on {t.device}, the call is on {device}")


def _required(device, dtype, **tensors):
    """As _check_tensors, of tensors that have to be given."""
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} must be a device tensor")
    _check_tensors(device, dtype, **tensors)


def _at(t):
    return None if t is None else t.data_ptr()


def _on_stream(fn):
    """Adds the keyword ``stream``: the whole call runs on it, what it allocates too, so that memory is not handed to
    another stream's work while the kernels still use it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        # all tensors of a call are on one device (checked there), so the first one speaks for them
        given = (t for x in (*args, *kwargs.values()) for t in (x if isinstance(x, (list, tuple)) else (x,)))
        first = next((t for t in given if isinstance(t, torch.Tensor)), None)
        if first is not None and first.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {first.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return call


def _call(fn, args, device):
    """Launches on the tensors' device (the library uses the current one) and its current stream."""
    lib = load_library()
    index = device.index
    s = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        status = getattr(lib, fn)(*args, s)
    else:
        with torch.cuda.device(device):
            status = getattr(lib, fn)(*args, s)
    if status != 0:
        _check(lib, fn, status)


def _heads(q, k, v, g):
    """Checks q, k [..., Hk, Dk], v [..., H, Dv] and g [..., H] or [H]; returns (H, Hk, Dk, Dv, g_per_head)."""
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a device tensor")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    _dev(q, "q")
    _check_tensors(q.device, dtype, k=k, v=v)
    _check_tensors(q.device, torch.float32, g=g)
    qs, vs = q.shape, v.shape
    if k.shape != qs:
        raise ValueError(f"k must have q's shape {tuple(qs)}, got {tuple(k.shape)}")
    if len(vs) != len(qs) or len(qs) < 3 or vs[:-2] != qs[:-2]:
        raise ValueError(f"v must be [..., H, Dv] over q's leading axes {tuple(qs[:-2])}, got {tuple(vs)}")
    H, Hk = vs[-2], qs[-2]
    if Hk < 1 or H < 1 or H % Hk != 0:
        raise ValueError(f"v's {H} heads must be a multiple of q's {Hk}")
    per_head = g.dim() == 1
    if (g.shape[0] != H) if per_head else (g.shape != vs[:-1]):
        raise ValueError(f"g must be [H] = [{H}] or {tuple(vs[:-1])}, got {tuple(g.shape)}")
    return H, Hk, qs[-1], vs[-1], per_head


def _sequences(q, v, cu_seqlens):
    """(B, T, N) of q [B, T, Hk, Dk], or with cu_seqlens of [T, Hk, Dk] (a leading 1 allowed)."""
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError(f"q must be [B, T, Hk, Dk], got {tuple(q.shape)}")
        return q.shape[0], q.shape[1], q.shape[0]
    _check_tensors(q.device, torch.int32, cu_seqlens=cu_seqlens)
    if q.dim() not in (3, 4) or (q.dim() == 4 and q.shape[0] != 1):
        raise ValueError(f"with cu_seqlens q must be [T, Hk, Dk], got {tuple(q.shape)}")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError(f"cu_seqlens must be [N + 1] with N >= 1, got {tuple(cu_seqlens.shape)}")
    return 1, q.shape[-3], cu_seqlens.shape[0] - 1


def _state(t, name, shape, device):
    if t is not None:
        _check_tensors(device, torch.float32, **{name: t})
        if t.shape != shape:
            raise ValueError(f"{name} must be [N, H, Dk, Dv] = {shape}, got {tuple(t.shape)}")


def _like(t, name, ref):
    """An output: allocated like ref when not given, checked when given."""
    if t is None:
        return torch.empty_like(ref)
    _check_tensors(ref.device, ref.dtype, **{name: t})
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have shape {tuple(ref.shape)}, got {tuple(t.shape)}")
    return t


def _workspace(fn, a, workspace, device):
    """Sets the workspace the call needs (allocated when not given); returns it so that it outlives the call."""
    need = _need(fn, a)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is not None:
        _check_tensors(device, None, workspace=workspace)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return workspace


@_on_stream
def linear_chunk_fwd(q, k, v, g, *, scale: float = 1.0, cu_seqlens=None, initial_state=None,
                     output_final_state: bool = True, out=None, final_state=None, workspace=None,
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
        _check_tensors(dev, torch.float32, checkpoints=checkpoints)
        if (checkpoints.dim() != 5 or checkpoints.shape[0] != N or checkpoints.shape[1] < 1
                or tuple(checkpoints.shape[2:]) != shape[1:] or checkpoint_every < 1):
            raise ValueError(f"checkpoints must be [N, slots >= 1, H, Dk, Dv] with N, H, Dk, Dv = {shape} and "
                             f"checkpoint_every >= 1; got {tuple(checkpoints.shape)}, every={checkpoint_every}")
        slots = checkpoints.shape[1]
    a = LinearFwdArgs(B, T, H, Hk, Dk, Dv, _DTYPES[q.dtype], _at(q), _at(k), _at(v), _at(g), per_head, scale,
                      _at(cu_seqlens), N, _at(initial_state), _at(out), _at(final_state), None, 0,
                      _at(checkpoints), checkpoint_every if slots else 0, slots)
    workspace = _workspace("kda_linear_chunk_fwd_workspace_size", a, workspace, dev)
    _call("kda_linear_chunk_fwd", (ctypes.byref(a),), dev)
    return out, final_state


@_on_stream
def linear_chunk_bwd(q, k, v, g, d_o, *, scale: float = 1.0, cu_seqlens=None, initial_state=None, dfinal_state=None,
                     need_dg: bool = True, dq=None, dk=None, dv=None, dg=None, dinitial_state=None, workspace=None):
    """Gradients of :func:`linear_chunk_fwd` (``kda_linear_chunk_bwd``) for the same arguments, given ``d_o`` (shaped
    like o, in its dtype) and ``dfinal_state`` ([N, H, Dk, Dv] fp32, None: zeros).  Returns (dq, dk, dv, dg, dinitial_state):
    the first three shaped and typed like q, k, v; dg fp32 shaped like g (None without ``need_dg``).  With ``need_dg`` dq and
    dk of bf16 calls take the state unrounded, without it rounded once, so their last bits differ."""
    H, Hk, Dk, Dv, per_head = _heads(q, k, v, g)
    B, T, N = _sequences(q, v, cu_seqlens)
    dev, shape = q.device, (N, H, Dk, Dv)
    _required(dev, q.dtype, d_o=d_o)
    if d_o.shape != v.shape:
        raise ValueError(f"d_o must have v's shape {tuple(v.shape)}, got {tuple(d_o.shape)}")
    _state(initial_state, "initial_state", shape, dev)
    _state(dfinal_state, "dfinal_state", shape, dev)
    dq, dk, dv = _like(dq, "dq", q), _like(dk, "dk", k), _like(dv, "dv", v)
    dg = _like(dg, "dg", g) if need_dg else None
    if dinitial_state is None:
        dinitial_state = torch.empty(shape, dtype=torch.float32, device=dev)
    _state(dinitial_state, "dinitial_state", shape, dev)
    a = LinearBwdArgs(B, T, H, Hk, Dk, Dv, _DTYPES[q.dtype], _at(q), _at(k), _at(v), _at(g), per_head, scale,
                      _at(cu_seqlens), N, _at(initial_state), _at(d_o), _at(dfinal_state), _at(dq), _at(dk),
                      _at(dv), _at(dg), _at(dinitial_state), None, 0)
    workspace = _workspace("kda_linear_chunk_bwd_workspace_size", a, workspace, dev)
    _call("kda_linear_chunk_bwd", (ctypes.byref(a),), dev)
    return dq, dk, dv, dg, dinitial_state


def linear_chunk_fwd_workspace_size(q, v, *, cu_seqlens=None) -> int:
    """Workspace bytes :func:`linear_chunk_fwd` needs for q [B, T, Hk, Dk] (or [T, Hk, Dk] with cu_seqlens) and v."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, T, N = _sequences(q, v, cu_seqlens)
    a = LinearFwdArgs(B, T, v.shape[-2], q.shape[-2], q.shape[-1], v.shape[-1], _DTYPES[q.dtype], scale=1.0,
                      cu_seqlens=_at(cu_seqlens), N=N)
    return _need("kda_linear_chunk_fwd_workspace_size", a)


def linear_chunk_bwd_workspace_size(q, v, *, cu_seqlens=None, g_per_head: bool = False, need_dg: bool = True,
                                    dfinal_state: bool = False) -> int:
    """Workspace bytes :func:`linear_chunk_bwd` needs; the flags say whether g is [H], whether dg is wanted and whether
    dfinal_state is given."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    B, T, N = _sequences(q, v, cu_seqlens)
    a = LinearBwdArgs(B, T, v.shape[-2], q.shape[-2], q.shape[-1], v.shape[-1], _DTYPES[q.dtype], scale=1.0,
                      cu_seqlens=_at(cu_seqlens), N=N, g_per_head=g_per_head)
    a.dg = 16 if need_dg else None             # only whether they are given is read
    a.d_final_state = 16 if dfinal_state else None
    return _need("kda_linear_chunk_bwd_workspace_size", a)


def _need(fn, a) -> int:
    lib = load_library()
    need = ctypes.c_size_t(0)
    _check(lib, fn, getattr(lib, fn)(ctypes.byref(a), ctypes.byref(need)))
    return need.value


@_on_stream
def linear_recurrent_step(q, k, v, g, state, *, scale: float = 1.0, slots=None, new_state=None, out=None):
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
    N, dev = q.shape[0], q.device
    _required(dev, torch.float32, state=state)
    _check_tensors(dev, torch.float32, new_state=new_state)
    shape = state.shape
    if len(shape) != 4 or shape[1] != H or shape[2] != Dk or shape[3] != Dv:
        raise ValueError(f"state must be [n_slots, H, Dk, Dv] with H, Dk, Dv = {(H, Dk, Dv)}, got {tuple(shape)}")
    if slots is not None:
        _check_tensors(dev, torch.int32, slots=slots)
        if slots.dim() != 1 or slots.shape[0] != N:
            raise ValueError(f"slots must be [N] = [{N}], got {tuple(slots.shape)}")
    if new_state is None:
        new_state = state
    elif new_state.shape != shape:
        raise ValueError(f"new_state must have state's shape {tuple(shape)}, got {tuple(new_state.shape)}")
    out = _like(out, "out", v)
    a = LinearStepArgs(N, H, Hk, Dk, Dv, _DTYPES[q.dtype], q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                       per_head, scale, _at(slots), shape[0], state.data_ptr(), new_state.data_ptr(), out.data_ptr())
    _call("kda_linear_recurrent_step", (ctypes.byref(a),), dev)
    return out
