"""Embedding table and gradients of a training step on packed streams
(include/thd_params.h).

``embedding`` takes the token ids as ``pack`` writes them, ``embedding_backward``
is its gradient with respect to the table, summed in a fixed order.
``clip_gradients`` scales a model's gradients down to a largest norm over all of
them; ``gradient_norm`` is that norm by itself, to be joined over ranks first.

Tables and rows are bfloat16, float16 or float32.  Calls return a device ``status``
word (int32 [1]) to look at when the host next waits.  A call runs on ``stream`` (the
current one if none is given), on which its outputs are allocated too; work that made
its inputs on another stream has to be ordered before it, and they have to live until
it is done.
"""

from __future__ import annotations

import operator

import numpy as np
import torch

from . import binding as _b
from .losses import _DTYPES, _F32, _I32, _I64, _U8, _address, _need_gpu, _run, _workspace

_Tensor = torch.Tensor
_dtype_of = operator.attrgetter("dtype")


def _matrix(x, name, width=None):
    """[rows, width] with contiguous rows at any stride; leading dimensions are
    flattened where that takes no copy."""
    if x is None:
        raise ValueError(f"{name} is required")
    if x.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    if x.dim() < 2:
        raise ValueError(f"{name} must be [rows, width]")
    if x.dim() > 2:
        try:
            x = x.view(-1, x.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: the leading dimensions cannot be flattened without a copy") from None
    if x.shape[1] < 1:
        raise ValueError(f"{name} needs at least one column")
    if width is not None and x.shape[1] != width:
        raise ValueError(f"{name} must have rows of {width} elements, got {x.shape[1]}")
    if not x.is_contiguous():
        if x.shape[1] > 1 and x.stride(1) != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        if x.shape[0] > 1 and x.stride(0) < x.shape[1]:
            raise ValueError(f"{name}: rows must not overlap")
    return x


def _stride(x) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def embedding(ids, table, mask=None, scale=1.0, out=None, stream=None):
    """``scale * table[ids]`` in the table's dtype: (rows [*ids.shape, width], status).
    ``ids`` int64, ``mask`` uint8 of the same number of elements or None: rows with
    mask 0 are 0."""
    if table is not None and table.dim() != 2:
        raise ValueError("table must be [vocab, width]")
    w = _matrix(table, "table")
    vocab, width = w.shape
    on = w.get_device()
    if ids is None:
        raise ValueError("ids is required")
    rows = ids.numel()
    ids_at = _address(ids, "ids", _I64, rows, on, True)
    mask_at = _address(mask, "mask", _U8, rows, on)
    _need_gpu(w, "table")
    to = None
    if out is not None:
        to = _matrix(out, "out", width)
        if out.dtype != w.dtype or out.device != w.device or to.shape[0] != rows:
            raise ValueError(f"out must be {w.dtype} [{rows}, {width}] on {w.device}")
    lib = _b.library()

    def call(handle):
        result = torch.empty((*ids.shape, width), dtype=w.dtype, device=w.device) if out is None else out
        x = to if to is not None else result.view(rows, width)
        status = torch.empty(1, dtype=_I32, device=w.device)
        code = lib.thd_embedding(ids_at, mask_at, rows, w.data_ptr(), _DTYPES[w.dtype], vocab, width, _stride(w),
                                 scale, x.data_ptr(), _stride(x), status.data_ptr(), handle)
        if code < 0:
            raise _b.ThdError(code, "thd_embedding")
        if out is not None:
            torch.autograd.graph.increment_version(out)
        return result, status
    return _run(call, stream)


def embedding_backward(drows, ids, vocab, mask=None, scale=1.0, out=None, accumulate=False, stream=None):
    """Gradient of ``(drows * embedding(ids, table)).sum()`` with respect to the table:
    (dtable [vocab, width], status).  ``out`` receives it where one is given, in the rows'
    dtype or float32; with ``accumulate`` it is added to what ``out`` holds."""
    x = _matrix(drows, "drows")
    rows, width = x.shape
    on = x.get_device()
    ids_at = _address(ids, "ids", _I64, rows, on, True)
    mask_at = _address(mask, "mask", _U8, rows, on)
    _need_gpu(x, "drows")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if out is not None:
        if out.dim() != 2:
            raise ValueError("out must be [vocab, width]")
        _matrix(out, "out", width)
        if out.dtype not in (x.dtype, _F32) or out.device != x.device or out.shape[0] != vocab:
            raise ValueError(f"out must be {x.dtype} or float32 [{vocab}, {width}] on {x.device}")
    lib = _b.library()

    def call(handle):
        dev = x.device
        grad = torch.empty((vocab, width), dtype=x.dtype, device=dev) if out is None else out
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_embedding_workspace_bytes(rows, vocab, width)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_embedding_backward(x.data_ptr(), _DTYPES[x.dtype], ids_at, mask_at, rows, vocab, width,
                                          _stride(x), scale, int(bool(accumulate)), grad.data_ptr(),
                                          _DTYPES[grad.dtype], _stride(grad), status.data_ptr(), room_at, nbytes,
                                          handle)
        if code < 0:
            raise _b.ThdError(code, "thd_embedding_backward")
        if out is not None:
            torch.autograd.graph.increment_version(out)
        return grad, status
    return _run(call, stream)


def _tensors(tensors, name, device):
    """Host arrays (addresses, elements, types) of contiguous tensors on one device."""
    try:
        dtypes = list(map(_dtype_of, tensors))
    except AttributeError:
        i = next(i for i, t in enumerate(tensors) if not isinstance(t, _Tensor))
        raise ValueError(f"{name}[{i}] must be a tensor, got {type(tensors[i]).__name__}") from None
    # one look at all of them; the one that is wrong is found only where there is one
    if not _DTYPES.keys() >= set(dtypes):
        i = next(i for i, d in enumerate(dtypes) if d not in _DTYPES)
        raise ValueError(f"{name}[{i}] must be bfloat16, float16 or float32, got {dtypes[i]}")
    on = list(map(_Tensor.get_device, tensors))
    if on.count(device) != len(on):
        i = next(i for i, d in enumerate(on) if d != device)
        raise ValueError(f"{name}[{i}] is on {tensors[i].device}, which is not the current device")
    whole = list(map(_Tensor.is_contiguous, tensors))
    if not all(whole):
        raise ValueError(f"{name}[{whole.index(False)}] must be contiguous")
    n = len(dtypes)
    return (np.fromiter(map(_Tensor.data_ptr, tensors), np.uint64, n),
            np.fromiter(map(_Tensor.numel, tensors), np.int64, n),
            np.fromiter(map(_DTYPES.__getitem__, dtypes), np.int32, n))


def _gradients(grads):
    grads = list(grads)
    if not torch.cuda.is_available():
        raise ValueError("gradients must live on the GPU")
    device = torch.cuda.current_device()
    at, elements, types = _tensors(grads, "grads", device)
    if len(at) > _b.THD_MAX_TENSORS:
        raise ValueError(f"at most {_b.THD_MAX_TENSORS} gradients, got {len(at)}")
    return grads, device, at, elements, types


def gradient_norm(grads, scale=1.0, stream=None):
    """``|scale|`` times the 2-norm of all elements of all tensors: (norm float32 [1],
    status)."""
    grads, device, at, elements, types = _gradients(grads)
    lib = _b.library()

    def call(handle):
        norm = torch.empty(1, dtype=_F32, device=device)
        status = torch.empty(1, dtype=_I32, device=device)
        nbytes = lib.thd_gradients_workspace_bytes(len(at))
        room, room_at = _workspace(nbytes, device)
        code = lib.thd_gradient_norm(at.ctypes.data, elements.ctypes.data, types.ctypes.data, len(at), scale,
                                     norm.data_ptr(), status.data_ptr(), room_at, nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_gradient_norm")
        return norm, status
    return _run(call, stream)


def clip_gradients(grads, max_norm, scale=1.0, outs=None, norm=None, stream=None):
    """Scales every gradient by ``scale * min(1, max_norm / (norm + 1e-6))``, in place or
    into ``outs`` (each of its gradient's dtype, or float32): (norm float32 [1], status).
    ``norm`` is that of all gradients, ``scale`` included, unless one is given (float32
    [1], e.g. joined over ranks).  A norm that is not finite makes every gradient 0 and
    sets the status word to THD_ERR_NORM."""
    grads, device, at, elements, types = _gradients(grads)
    out_at, out_types = at, types
    if outs is not None:
        outs = list(outs)
        out_at, out_elements, out_types = _tensors(outs, "outs", device)
        if len(outs) != len(grads) or not np.array_equal(out_elements, elements):
            raise ValueError("outs and grads differ in number or size")
        wrong = (out_types != types) & (out_types != _b.THD_FP32)
        if wrong.any():
            i = int(np.argmax(wrong))
            raise ValueError(f"outs[{i}] must be {grads[i].dtype} or float32, got {outs[i].dtype}")
    norm_at = _address(norm, "norm", _F32, 1, device)
    lib = _b.library()

    def call(handle):
        result = torch.empty(1, dtype=_F32, device=device)
        status = torch.empty(1, dtype=_I32, device=device)
        nbytes = 0 if norm is not None else lib.thd_gradients_workspace_bytes(len(at))
        room, room_at = _workspace(nbytes, device)
        code = lib.thd_clip_gradients(at.ctypes.data, out_at.ctypes.data, elements.ctypes.data, types.ctypes.data,
                                      out_types.ctypes.data, len(at), max_norm, scale, norm_at, result.data_ptr(),
                                      status.data_ptr(), room_at, nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_clip_gradients")
        torch.autograd.graph.increment_version(grads if outs is None else outs)
        return result, status
    return _run(call, stream)
