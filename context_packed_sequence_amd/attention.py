"""Attention inside the documents of a packed stream, with its gradient
(include/thd_attention.h).

Queries are the rows of the whole stream or of one context-parallel rank's
zigzag share, keys and values the whole stream in token order.  Tensors are
[rows, heads, dim] in bfloat16 or float16 with contiguous heads; rows and heads
may be strided, as in views of one projection's output.  Gradients are returned
by a call of their own rather than through autograd, as the losses' are:
``out.backward(dout)`` of a model is ``packed_attention_backward(dout, ...)``.

Calls return a device ``status`` word (int32 [1]) to look at when the host next
waits.  A call runs on ``stream`` (the current one if none is given), on which its
outputs are allocated too; work that made its inputs on another stream has to be
ordered before it, and they have to live until it is done.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import binding as _b
from .losses import _address, _need_gpu, _run, _workspace

_DTYPES = {torch.bfloat16: _b.THD_BF16, torch.float16: _b.THD_FP16}
_I32, _F32 = torch.int32, torch.float32


def _heads(x, name, rows=None, heads=None, like=None):
    """The tensor as the library takes it, after the checks it cannot make."""
    if x is None:
        raise ValueError(f"{name} is required")
    if x.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16 or float16, got {x.dtype}")
    if x.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, dim]")
    if like is not None:
        if x.dtype != like.dtype:
            raise ValueError(f"{name} must be {like.dtype}, got {x.dtype}")
        if x.get_device() != like.get_device():
            raise ValueError(f"{name} must be on {like.device}, got {x.device}")
        if x.shape[2] != like.shape[2]:
            raise ValueError(f"{name} must have heads of {like.shape[2]} elements, got {x.shape[2]}")
    if (rows is not None and x.shape[0] != rows) or (heads is not None and x.shape[1] != heads):
        raise ValueError(f"{name} must be [{rows}, {x.shape[1] if heads is None else heads}, {x.shape[2]}], "
                         f"got {list(x.shape)}")
    if x.numel() and x.stride(2) != 1 and x.shape[2] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    rows_apart = x.stride(0) if x.shape[0] > 1 else x.shape[1] * x.shape[2]
    heads_apart = x.stride(1) if x.shape[1] > 1 else x.shape[2]
    if rows_apart % 8 or heads_apart % 8 or x.data_ptr() % 16:
        raise ValueError(f"{name}: rows and heads must start at multiples of 16 bytes")
    if x.shape[0] > 1 and rows_apart < x.shape[2]:
        raise ValueError(f"{name}: rows must not overlap")
    return _b.thd_heads(x.data_ptr() if x.numel() else None, rows_apart, heads_apart)


def _shape(q, k, v, cu_seqlens_padded, cu_seqlens, causal, window, scale, cap, cp_size, rank):
    """(shape, q, k, v as the library takes them)"""
    q_at = _heads(q, "q")
    k_at = _heads(k, "k", like=q)
    tokens, kv_heads, dim = k.shape
    v_at = _heads(v, "v", tokens, kv_heads, like=q)
    rows, heads = q.shape[:2]
    if dim % 8 or not 8 <= dim <= _b.THD_MAX_HEAD_DIM:
        raise ValueError(f"heads must have a multiple of 8 elements, 8 to {_b.THD_MAX_HEAD_DIM}, got {dim}")
    if kv_heads < 1 or heads < 1 or heads % kv_heads:
        raise ValueError(f"the query heads must be a multiple of the key heads, got {heads} and {kv_heads}")
    if not 1 <= cp_size <= _b.THD_MAX_CP or not 0 <= rank < cp_size:
        raise ValueError(f"rank {rank} of {cp_size} is none")
    if rows * cp_size != tokens:
        raise ValueError(f"q must have {tokens} / {cp_size} rows, got {rows}")
    if window < 0:
        raise ValueError("window must not be negative (0: none)")
    if cu_seqlens_padded is None or cu_seqlens_padded.numel() < 1:
        raise ValueError("cu_seqlens_padded needs at least one boundary")
    n_slots = cu_seqlens_padded.numel() - 1
    on = q.get_device()
    padded_at = _address(cu_seqlens_padded, "cu_seqlens_padded", _I32, n_slots + 1, on)
    real_at = _address(cu_seqlens, "cu_seqlens", _I32, n_slots + 1, on)
    _need_gpu(q, "q")
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    shape = _b.thd_attention_shape(_DTYPES[q.dtype], heads, kv_heads, dim, int(bool(causal)), min(window, 2 ** 31 - 1),
                                   cp_size, rank, n_slots, tokens, scale, cap or 0.0, padded_at, real_at)
    return shape, q_at, k_at, v_at


def packed_attention(q, k, v, cu_seqlens_padded, cu_seqlens=None, causal=True, window=0, scale=None, cap=0.0,
                     cp_size=1, rank=0, out=None, stream=None):
    """Attention of each query row over its own document: (out [rows, heads, dim],
    lse float32 [heads, rows], status).

    ``q`` [tokens / cp_size, heads, dim] are the whole stream's queries, or the rows
    that ``rank`` of ``cp_size`` holds in zigzag order; ``k`` and ``v`` [tokens,
    kv_heads, dim] the whole stream in token order.  ``window`` w lets position i see
    positions closer than w, ``cap`` c replaces a score z by c tanh(z / c),
    ``scale`` is 1 / sqrt(dim) unless given.  Pads, by ``cu_seqlens`` (real
    boundaries), take no part; their rows of ``out`` are 0, their lse -inf."""
    shape, q_at, k_at, v_at = _shape(q, k, v, cu_seqlens_padded, cu_seqlens, causal, window, scale, cap, cp_size, rank)
    if out is not None:
        _heads(out, "out", q.shape[0], q.shape[1], like=q)
    lib = _b.library()

    def call(handle):
        dev = q.device
        result = torch.empty(q.shape, dtype=q.dtype, device=dev) if out is None else out
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=_F32, device=dev)
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_attention_workspace_bytes(ctypes.byref(shape), 0)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_attention(ctypes.byref(shape), ctypes.byref(q_at), ctypes.byref(k_at), ctypes.byref(v_at),
                                 ctypes.byref(_heads(result, "out")), lse.data_ptr(), status.data_ptr(), room_at,
                                 nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_attention")
        if out is not None:
            torch.autograd.graph.increment_version(out)
        return result, lse, status
    return _run(call, stream)


def packed_attention_backward(dout, q, k, v, out, lse, cu_seqlens_padded, cu_seqlens=None, causal=True, window=0,
                              scale=None, cap=0.0, cp_size=1, rank=0, grads=None, stream=None):
    """Gradients of ``(dout * out).sum()``: (dq, dk, dv, status), in the shapes of
    q, k and v.  ``out`` and ``lse`` are what ``packed_attention`` returned for the same
    arguments.  With ``cp_size`` above 1, dk and dv are this rank's part of a sum over the
    ranks.  ``grads`` may give the three tensors to write, e.g. views of one
    projection's gradient."""
    shape, q_at, k_at, v_at = _shape(q, k, v, cu_seqlens_padded, cu_seqlens, causal, window, scale, cap, cp_size, rank)
    rows, heads = q.shape[:2]
    out_at = _heads(out, "out", rows, heads, like=q)
    dout_at = _heads(dout, "dout", rows, heads, like=q)
    if lse is not None and tuple(lse.shape) != (heads, rows):
        raise ValueError(f"lse must be [{heads}, {rows}], got {list(lse.shape)}")
    lse_at = _address(lse, "lse", _F32, heads * rows, q.get_device(), True)
    if grads is not None:
        if len(grads) != 3:
            raise ValueError("grads must be three tensors, for q, k and v")
        for name, g, x in zip(("dq", "dk", "dv"), grads, (q, k, v)):
            _heads(g, name, x.shape[0], x.shape[1], like=q)
    lib = _b.library()

    def call(handle):
        dev = q.device
        dq, dk, dv = grads if grads is not None else [torch.empty(x.shape, dtype=x.dtype, device=dev)
                                                      for x in (q, k, v)]
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_attention_workspace_bytes(ctypes.byref(shape), 1)
        room, room_at = _workspace(nbytes, dev)
        at = [ctypes.byref(x) for x in (q_at, k_at, v_at, out_at)]
        to = [ctypes.byref(_heads(x, "gradient")) for x in (dq, dk, dv)]
        code = lib.thd_attention_backward(ctypes.byref(shape), *at, lse_at, ctypes.byref(dout_at), *to,
                                          status.data_ptr(), room_at, nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_attention_backward")
        if grads is not None:
            for g in grads:
                torch.autograd.graph.increment_version(g)
        return dq, dk, dv, status
    return _run(call, stream)
