"""Binding of the linear-attention entry points: layers with a decay for each
head, beside a hybrid model's GDN layers and over the same kind of state slots.

Argument marshalling only: dtypes, devices, shapes and strides are checked here,
then the C ABI of ``include/gdn.h`` runs on the current torch stream (or the one
given).
"""
from __future__ import annotations

import ctypes
import struct

from . import GdnError, lib
from .attention import _HEADS, _at, _at_or_none, _gpu, _heads_layout, _launch, _refuse, _torch

EXPORTS = ("lin_attn_step", "lin_attn_step_tokens", "lin_attn_prefill", "lin_attn_prefill_workspace_bytes")

_P, _i32, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float


class LinDims(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("B", "T", "H_k", "H_v", "d_k", "d_v", "N", "per_token")]


_DIMS = struct.Struct("8i")
assert _DIMS.size == ctypes.sizeof(LinDims)


def declare(L) -> None:
    """Argument types of this module's entry points (structures go as pointers or as packed bytes)."""
    size = ctypes.c_size_t
    for name, args, res in (
            ("lin_attn_step", [_P] * 9 + [_f32, _P], _i32),
            ("lin_attn_step_tokens", [_P] * 9 + [_f32, _P], _i32),
            ("lin_attn_prefill_workspace_bytes", [_P], size),
            ("lin_attn_prefill", [_P] * 10 + [_f32, _P, size, _P], _i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


# ------------------------------------------------------------------ checks

def _state_layout(state):
    s = state.shape
    if len(s) != 4:
        raise ValueError("state must be [N][H_v][d_k][d_v]")
    return s


def _rows(t, name, B, T, H, d, dtype, dev):
    """[B][T][H][d] whose tokens lie a fixed stride apart, as the C structure."""
    s, step = t.shape, t.stride()
    if len(s) != 4 or s != (B, T, H, d):
        raise ValueError(f"{name} must be [{B}][{T}][{H}][{d}], got {list(s)}")
    if step[3] != 1:
        raise ValueError(f"{name}: the head's values must be contiguous")
    if B > 1 and T > 1 and step[0] != T * step[1]:
        raise ValueError(f"{name}: the rows' tokens must lie a fixed stride apart")
    if t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    # the stride of an axis of one says nothing, and torch lets it be anything
    return _HEADS.pack(t.data_ptr(), step[1] if T > 1 else (step[0] if B > 1 else 0), step[2] if H > 1 else 0)


def _packed(t, name, T, H, d, dtype, dev):
    """[T][H][d] as the C structure."""
    s, step = t.shape, t.stride()
    if s != (T, H, d) or step[2] != 1:
        _heads_layout(t, name, T, H, d)
    if t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    return _HEADS.pack(t.data_ptr(), step[0] if T > 1 else 0, step[1] if H > 1 else 0)


def _decays(g, shape, H_v):
    """Whether g has a decay for every token (shape, then [H_v]) or one a head ([H_v])."""
    s = tuple(g.shape)
    if s == (H_v,):
        return 0
    if s != shape + (H_v,):
        raise ValueError(f"g must be [{H_v}] or {list(shape) + [H_v]}, got {list(s)}")
    return 1


def _head_counts(q, axis, H_v):
    H_k = q.shape[axis] if q.dim() > axis else 0
    if H_k < 1 or H_v % H_k:
        raise ValueError(f"state has {H_v} heads, q {H_k}: the first must be a multiple of the second")
    return H_k


# ------------------------------------------------------------------ entry points

def _step(name, q, k, v, g, state, read_slot, slots, slots_name, slots_shape, out, q_scale, stream):
    torch = _torch()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N, H_v, d_k, d_v = _state_layout(state)
    if q.dim() != 4:
        raise ValueError(f"q must be [B][T][H_k][d_k], got {list(q.shape)}")
    B, T = q.shape[:2]
    H_k = _head_counts(q, 2, H_v)
    if read_slot.shape != (B,):
        raise ValueError("read_slot must be [B]")
    if slots is not None and slots.shape != (slots_shape(B, T)):
        raise ValueError(f"{slots_name} must be {list(slots_shape(B, T))}")
    per_token = _decays(g, (B, T), H_v)
    dev = _gpu(state, "state")
    _launch(name, getattr(lib(), name), dev, stream, _DIMS.pack(B, T, H_k, H_v, d_k, d_v, N, per_token),
            _rows(q, "q", B, T, H_k, d_k, bf, dev), _rows(k, "k", B, T, H_k, d_k, bf, dev),
            _rows(v, "v", B, T, H_v, d_v, bf, dev), _at(g, "g", f32, dev), _at(state, "state", f32, dev),
            _at(read_slot, "read_slot", i32, dev), _at_or_none(slots, slots_name, i32, dev),
            _rows(out, "out", B, T, H_v, d_v, bf, dev), q_scale)


def lin_attn_step(q, k, v, g, state, read_slot, write_slot, out, *, q_scale: float = 1.0, stream=None) -> None:
    """Linear attention with a decay for each head, one token a row or a few (see ``lin_attn_step`` in
    include/gdn.h).

    q and k [B][T][H_k][d_k], v and out [B][T][H_v][d_v] bf16 (views of a packed projection are fine, tokens a
    fixed stride apart), g the log decays [H_v] or [B][T][H_v] fp32, state [N][H_v][d_k][d_v] fp32,
    read_slot/write_slot [B] int32 (write_slot None => in place)."""
    _step("lin_attn_step", q, k, v, g, state, read_slot, write_slot, "write_slot", lambda B, T: (B,), out, q_scale,
          stream)


def lin_attn_step_tokens(q, k, v, g, state, read_slot, token_slots, out, *, q_scale: float = 1.0,
                         stream=None) -> None:
    """T tokens a row from the read slot, the state after token t kept in slot token_slots[r][t] (0: not kept);
    the read slot is not written (see ``lin_attn_step_tokens`` in include/gdn.h)."""
    if token_slots is None:
        raise ValueError("token_slots is required")
    _step("lin_attn_step_tokens", q, k, v, g, state, read_slot, token_slots, "token_slots", lambda B, T: (B, T), out,
          q_scale, stream)


def lin_attn_prefill_workspace_bytes(B: int, T: int, H_k: int, H_v: int, d_k: int, d_v: int) -> int:
    """The workspace lin_attn_prefill needs for up to B sequences of up to T tokens in all, in bytes, on the current
    GPU."""
    n = lib().lin_attn_prefill_workspace_bytes(_DIMS.pack(B, T, H_k, H_v, d_k, d_v, 1, 0))
    if n == 0:
        raise GdnError("lin_attn_prefill_workspace_bytes", 2)
    return n


def lin_attn_prefill(q, k, v, g, cu_seqlens, state, read_slot, write_slot, out, workspace, *, q_scale: float = 1.0,
                     stream=None) -> None:
    """Linear attention with a decay for each head over packed prompts (see ``lin_attn_prefill`` in
    include/gdn.h).

    q and k [T][H_k][d_k], v and out [T][H_v][d_v] bf16 by their strides, g the log decays [H_v] or [T][H_v]
    fp32, cu_seqlens [B+1], read_slot and write_slot [B] int32 (write_slot None => in place; a read slot of 0 with
    a write slot => from zeros), workspace a uint8 tensor of lin_attn_prefill_workspace_bytes."""
    torch = _torch()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N, H_v, d_k, d_v = _state_layout(state)
    if q.dim() != 3:
        raise ValueError(f"q must be [T][H_k][d_k], got {list(q.shape)}")
    T = q.shape[0]
    H_k = _head_counts(q, 1, H_v)
    s = read_slot.shape
    if len(s) != 1 or cu_seqlens.shape != (s[0] + 1,):
        raise ValueError("read_slot must be [B] and cu_seqlens [B+1]")
    B = s[0]
    if write_slot is not None and write_slot.shape != s:
        raise ValueError("write_slot must be [B]")
    per_token = _decays(g, (T,), H_v)
    dev = _gpu(state, "state")
    _launch("lin_attn_prefill", lib().lin_attn_prefill, dev, stream,
            _DIMS.pack(B, T, H_k, H_v, d_k, d_v, N, per_token), _packed(q, "q", T, H_k, d_k, bf, dev),
            _packed(k, "k", T, H_k, d_k, bf, dev), _packed(v, "v", T, H_v, d_v, bf, dev), _at(g, "g", f32, dev),
            _at(cu_seqlens, "cu_seqlens", i32, dev), _at(state, "state", f32, dev),
            _at(read_slot, "read_slot", i32, dev), _at_or_none(write_slot, "write_slot", i32, dev),
            _packed(out, "out", T, H_v, d_v, bf, dev), q_scale, _at(workspace, "workspace", torch.uint8, dev),
            workspace.numel())
