"""Linear attention with a decay for each head (``kda_linear_*``).

The recurrence next to KDA's that writes without the delta rule and forgets with
one scalar per head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DTYPES, LinearStepArgs, _check, _dev, _ptr, _stream, load_library


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
