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
_byref = ctypes.byref


def _heads(x, name, rows=None, heads=None, like=None):
    """The tensor as the library takes it, after the checks it cannot make."""
    if x is None:
        raise ValueError(f"{name} is required")
    dtype, sizes = x.dtype, x.shape
    if dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16 or float16, got {dtype}")
    if len(sizes) != 3:
        raise ValueError(f"{name} must be [rows, heads, dim]")
    n, m, dim = sizes
    if like is not None:
        if dtype != like.dtype:
            raise ValueError(f"{name} must be {like.dtype}, got {dtype}")
        if x.get_device() != like.get_device():
            raise ValueError(f"{name} must be on {like.device}, got {x.device}")
        if dim != like.shape[2]:
            raise ValueError(f"{name} must have heads of {like.shape[2]} elements, got {dim}")
    if (rows is not None and n != rows) or (heads is not None and m != heads):
        raise ValueError(f"{name} must be [{rows}, {m if heads is None else heads}, {dim}], got {list(sizes)}")
    rows_apart, heads_apart, step = x.stride()
    some = n and m and dim
    if some and step != 1 and dim != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if n <= 1:
        rows_apart = m * dim
    if m <= 1:
        heads_apart = dim
    at = x.data_ptr()
    if rows_apart % 8 or heads_apart % 8 or at % 16:
        raise ValueError(f"{name}: rows and heads must start at multiples of 16 bytes")
    if n > 1 and rows_apart < dim:
        raise ValueError(f"{name}: rows must not overlap")
    return _b.thd_heads(at if some else None, rows_apart, heads_apart)


def _shape(q, k, v, cu_seqlens_padded, cu_seqlens, causal, window, scale, cap, cp_size, rank):
    """(shape, q, k, v as the library takes them)"""
    q_at = _heads(q, "q")
    k_at = _heads(k, "k", like=q)
    tokens, kv_heads, dim = k.shape
    v_at = _heads(v, "v", tokens, kv_heads, like=q)
    rows, heads, _ = q.shape
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
    rows, heads, dim = q.shape
    out_at = None if out is None else _heads(out, "out", rows, heads, like=q)
    lib = _b.library()

    def call(handle):
        dev = q.device
        result, result_at = out, out_at
        if out is None:
            result = torch.empty((rows, heads, dim), dtype=q.dtype, device=dev)
            result_at = _b.thd_heads(result.data_ptr(), heads * dim, dim)
        lse = torch.empty((heads, rows), dtype=_F32, device=dev)
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_attention_workspace_bytes(_byref(shape), 0)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_attention(_byref(shape), _byref(q_at), _byref(k_at), _byref(v_at), _byref(result_at),
                                 lse.data_ptr(), status.data_ptr(), room_at, nbytes, handle)
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
    rows, heads, _ = q.shape
    out_at = _heads(out, "out", rows, heads, like=q)
    dout_at = _heads(dout, "dout", rows, heads, like=q)
    if lse is not None and tuple(lse.shape) != (heads, rows):
        raise ValueError(f"lse must be [{heads}, {rows}], got {list(lse.shape)}")
    lse_at = _address(lse, "lse", _F32, heads * rows, q.get_device(), True)
    if grads is not None:
        if len(grads) != 3:
            raise ValueError("grads must be three tensors, for q, k and v")
        to = [_heads(g, name, x.shape[0], x.shape[1], like=q)
              for name, g, x in zip(("dq", "dk", "dv"), grads, (q, k, v))]
    lib = _b.library()

    def call(handle):
        dev = q.device
        results, at = grads, None if grads is None else to
        if grads is None:
            results = [torch.empty(x.shape, dtype=x.dtype, device=dev) for x in (q, k, v)]
            at = [_b.thd_heads(g.data_ptr(), g.shape[1] * g.shape[2], g.shape[2]) for g in results]
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_attention_workspace_bytes(_byref(shape), 1)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_attention_backward(_byref(shape), _byref(q_at), _byref(k_at), _byref(v_at), _byref(out_at),
                                          lse_at, _byref(dout_at), _byref(at[0]), _byref(at[1]), _byref(at[2]),
                                          status.data_ptr(), room_at, nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_attention_backward")
        if grads is not None:
            for g in grads:
                torch.autograd.graph.increment_version(g)
        return (*results, status)
    return _run(call, stream)
