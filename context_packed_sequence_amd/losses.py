"""Losses on packed token streams, with their gradients (include/thd_loss.h).

Rows are token positions of a packed stream, in natural or zigzag order;
``labels`` and ``mask`` are what ``roll_labels`` and ``Route.roll_labels_zigzag``
write (``shifted[j - 1]`` and ``mask[j]`` for shift j), documents the slots of
``cu_seqlens_padded``.  The gradient is returned beside the loss rather than
through autograd: a model's backward starts from it with
``logits.backward(dlogits)``.

Logits are [rows, vocab] (leading dimensions are flattened where that takes no
copy) in bfloat16, float16 or float32, their last dimension contiguous; rows
may be strided, as in a view of the first columns of a padded vocabulary.  Every
call returns a device ``status`` word (int32 [1]) to look at when the host next
waits, and runs on ``stream`` (the current one if none is given), on which its
outputs are allocated too.
"""

from __future__ import annotations

import contextlib

import torch

from . import binding as _b

_DTYPES = {torch.bfloat16: _b.THD_BF16, torch.float16: _b.THD_FP16, torch.float32: _b.THD_FP32}


def _on(stream):
    """Outputs and workspaces belong to the stream that writes them: memory
    handed back to another stream's pool could be given out again too early."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _rows_of(logits, name="logits"):
    if logits.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {logits.dtype}")
    if logits.dim() < 2:
        raise ValueError(f"{name} must be [rows, vocab]")
    if logits.dim() > 2:
        try:
            logits = logits.view(-1, logits.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: the leading dimensions cannot be flattened without a copy") from None
    if logits.shape[1] < 1:
        raise ValueError(f"{name} needs at least one column")
    if logits.shape[1] > 1 and logits.stride(1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if logits.shape[0] > 1 and logits.stride(0) < logits.shape[1]:
        raise ValueError(f"{name}: rows must not overlap")
    return logits


def _stride(x) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _per_row(x, name, dtype, rows, device):
    if x is None:
        return
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if x.numel() != rows:
        raise ValueError(f"{name} must have {rows} elements, got {x.numel()}")
    if x.device != device:
        raise ValueError(f"{name} must be on {device}, got {x.device}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_gpu(x, name):
    if not x.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if x.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {x.device}, which is not the current device")


def _grad_rows(logits, out):
    """Where the gradient goes.  A new one has rows that start at the same place
    within 16 bytes as the logits' rows, which is the layout that is written
    fastest: contiguous for contiguous logits, else padded by a few columns."""
    if out is not None:
        if out.dtype != logits.dtype or out.device != logits.device:
            raise ValueError(f"out must be {logits.dtype} on {logits.device}")
        out = _rows_of(out, "out")
        if out.shape != logits.shape:
            raise ValueError(f"out must be {tuple(logits.shape)}, got {tuple(out.shape)}")
        return out
    rows, vocab = logits.shape
    size = logits.element_size()
    per = 16 // size
    lead = logits.data_ptr() % 16 // size
    pad = (_stride(logits) - vocab) % per
    if not lead and not pad:
        return torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    room = torch.empty(lead + rows * (vocab + pad), dtype=logits.dtype, device=logits.device)
    return room.as_strided((rows, vocab), (vocab + pad, 1), lead)


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _like(grad, x):
    """The gradient in the logits' own shape."""
    return grad if x.dim() == 2 else grad.unflatten(0, x.shape[:-1])


def token_logprobs(logits, labels, mask=None, stream=None):
    """Log-probability of each row's label and the row's log-sum-exp:
    (logp float32 [rows], lse float32 [rows], status)."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    dev = z.device
    if labels is None:
        raise ValueError("labels is required")
    _per_row(labels, "labels", torch.int64, rows, dev)
    _per_row(mask, "mask", torch.uint8, rows, dev)
    _need_gpu(z, "logits")
    dtype = _DTYPES[z.dtype]
    with _on(stream):
        logp = torch.empty(rows, dtype=torch.float32, device=dev)
        lse = torch.empty(rows, dtype=torch.float32, device=dev)
        status = torch.empty(1, dtype=torch.int32, device=dev)
        nbytes = _b.thd_loss_workspace_bytes(rows, vocab, dtype, 0)
        _b.thd_token_logprobs(z.data_ptr(), dtype, rows, vocab, _stride(z), labels, mask, logp, lse, status,
                              _workspace(nbytes, dev), nbytes, stream)
    return logp, lse, status


def token_logprobs_backward(dlogp, logits, labels, lse, mask=None, out=None, stream=None):
    """Gradient of ``(dlogp * logp).sum()`` with respect to the logits, in their
    dtype.  ``lse`` is what ``token_logprobs`` returned; ``out`` may be the
    logits themselves, which are then replaced."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    dev = z.device
    for name, x, dtype in (("dlogp", dlogp, torch.float32), ("labels", labels, torch.int64),
                           ("lse", lse, torch.float32)):
        if x is None:
            raise ValueError(f"{name} is required")
        _per_row(x, name, dtype, rows, dev)
    _per_row(mask, "mask", torch.uint8, rows, dev)
    _need_gpu(z, "logits")
    with _on(stream):
        grad = _grad_rows(z, out)
        _b.thd_token_logprobs_backward(dlogp, z.data_ptr(), _DTYPES[z.dtype], rows, vocab, _stride(z), labels, lse,
                                       mask, grad.data_ptr(), _stride(grad), stream)
    return _like(grad, logits) if out is None else out


def policy_loss(logits, labels, old_logp, advantages, mask=None, ref_logp=None, weights=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, out=None, stream=None):
    """Clipped policy loss with a KL term: (loss float32 [rows], logp float32
    [rows], dlogits, status).  ``loss`` holds each row's weighted term (its sum
    is the loss), ``dlogits`` the gradient of that sum; ``weights`` carries the
    normalisation, e.g. one over the number of labelled tokens."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    dev = z.device
    for name, x, dtype in (("labels", labels, torch.int64), ("old_logp", old_logp, torch.float32),
                           ("advantages", advantages, torch.float32)):
        if x is None:
            raise ValueError(f"{name} is required")
        _per_row(x, name, dtype, rows, dev)
    _per_row(mask, "mask", torch.uint8, rows, dev)
    _per_row(ref_logp, "ref_logp", torch.float32, rows, dev)
    _per_row(weights, "weights", torch.float32, rows, dev)
    if kl_coef and ref_logp is None:
        raise ValueError("a KL term needs ref_logp")
    _need_gpu(z, "logits")
    dtype = _DTYPES[z.dtype]
    with _on(stream):
        grad = _grad_rows(z, out)
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
        logp = torch.empty(rows, dtype=torch.float32, device=dev)
        status = torch.empty(1, dtype=torch.int32, device=dev)
        nbytes = _b.thd_loss_workspace_bytes(rows, vocab, dtype, 1)
        _b.thd_policy_loss(z.data_ptr(), dtype, rows, vocab, _stride(z), labels, mask, old_logp, ref_logp, advantages,
                           weights, clip_low, clip_high, kl_coef, loss, logp, grad.data_ptr(), _stride(grad), status,
                           _workspace(nbytes, dev), nbytes, stream)
    return loss, logp, _like(grad, logits) if out is None else out, status


def distill_topk(logits, teacher_logits, teacher_ids, mask=None, weights=None, temperature=1.0, out=None,
                 stream=None):
    """Distillation from a teacher's top logits: (loss float32 [rows], dlogits,
    status).  ``teacher_logits`` [rows, k] and ``teacher_ids`` [rows, k] (int32
    or int64; -1 leaves an entry out) are the teacher's largest logits and their
    columns."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    dev = z.device
    if teacher_logits is None or teacher_ids is None:
        raise ValueError("teacher_logits and teacher_ids are required")
    if teacher_ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"teacher_ids must be int32 or int64, got {teacher_ids.dtype}")
    t = _rows_of(teacher_logits, "teacher_logits")
    k = t.shape[1]
    if k > _b.THD_MAX_TOPK:
        raise ValueError(f"at most {_b.THD_MAX_TOPK} teacher columns, got {k}")
    for name, x in (("teacher_logits", t), ("teacher_ids", teacher_ids)):
        if x.numel() != rows * k or x.shape[-1] != k:
            raise ValueError(f"{name} must be [{rows}, {k}]")
        if x.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {x.device}")
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _per_row(mask, "mask", torch.uint8, rows, dev)
    _per_row(weights, "weights", torch.float32, rows, dev)
    _need_gpu(z, "logits")
    dtype = _DTYPES[z.dtype]
    with _on(stream):
        grad = _grad_rows(z, out)
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
        status = torch.empty(1, dtype=torch.int32, device=dev)
        nbytes = _b.thd_loss_workspace_bytes(rows, vocab, dtype, k)
        _b.thd_distill_topk(z.data_ptr(), dtype, rows, vocab, _stride(z), t.data_ptr(), _DTYPES[t.dtype],
                            teacher_ids.data_ptr(), teacher_ids.element_size(), k, k, mask, weights, temperature,
                            loss, grad.data_ptr(), _stride(grad), status, _workspace(nbytes, dev), nbytes, stream)
    return loss, _like(grad, logits) if out is None else out, status


def preference_loss(logp, ref_logp, pairs, cu_seqlens_padded, mask=None, beta=0.1, label_smoothing=0.0, scale=1.0,
                    stream=None):
    """Preference loss over pairs of documents of a packed stream in token
    order: (loss float32 [pairs], rewards float32 [pairs, 2], dlogp float32
    [tokens], status).  ``pairs`` int32 [pairs, 2] holds (chosen, rejected) slot
    numbers of ``cu_seqlens_padded``; ``scale`` multiplies every loss (one over
    the number of pairs for a mean).  ``dlogp`` goes to
    ``token_logprobs_backward``."""
    if logp is None or pairs is None or cu_seqlens_padded is None:
        raise ValueError("logp, pairs and cu_seqlens_padded are required")
    total = logp.numel()
    dev = logp.device
    _per_row(logp, "logp", torch.float32, total, dev)
    _per_row(ref_logp, "ref_logp", torch.float32, total, dev)
    _per_row(mask, "mask", torch.uint8, total, dev)
    _per_row(cu_seqlens_padded, "cu_seqlens_padded", torch.int32, cu_seqlens_padded.numel(), dev)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [pairs, 2]")
    n_pairs = pairs.shape[0]
    _per_row(pairs, "pairs", torch.int32, 2 * n_pairs, dev)
    if n_pairs > _b.THD_MAX_PAIRS:
        raise ValueError(f"at most {_b.THD_MAX_PAIRS} pairs, got {n_pairs}")
    n_slots = cu_seqlens_padded.numel() - 1
    if n_slots < 0:
        raise ValueError("cu_seqlens_padded needs at least one boundary")
    _need_gpu(logp, "logp")
    with _on(stream):
        loss = torch.empty(n_pairs, dtype=torch.float32, device=dev)
        rewards = torch.empty((n_pairs, 2), dtype=torch.float32, device=dev)
        dlogp = torch.empty(total, dtype=torch.float32, device=dev)
        status = torch.empty(1, dtype=torch.int32, device=dev)
        nbytes = _b.thd_preference_workspace_bytes(total, n_slots)
        _b.thd_preference_loss(logp, ref_logp, mask, cu_seqlens_padded, n_slots, total, pairs, n_pairs, beta,
                               label_smoothing, scale, loss, rewards, dlogp, status, _workspace(nbytes, dev), nbytes,
                               stream)
    return loss, rewards, dlogp, status
