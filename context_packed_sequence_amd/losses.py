"""Losses on packed token streams, with their gradients (include/thd_loss.h).

Rows are token positions of a packed stream, in natural or zigzag order;
``labels`` and ``mask`` are what ``roll_labels`` and ``Route.roll_labels_zigzag``
write (``shifted[j - 1]`` and ``mask[j]`` for shift j), documents the slots of
``cu_seqlens_padded``.  The gradient is returned beside the loss rather than
through autograd: a model's backward starts from it with
``logits.backward(dlogits)``.  ``out`` receives it where one is given; it may be
the logits themselves, as long as no earlier operation needs them for its own
backward (a cap by ``tanh`` does: autograd raises then).

Logits are [rows, vocab] (leading dimensions are flattened where that takes no
copy) in bfloat16, float16 or float32, their last dimension contiguous; rows
may be strided, as in a view of the first columns of a padded vocabulary.  The forward
calls return a device ``status`` word (int32 [1]) to look at when the host next
waits.  A call runs on ``stream`` (the current one if none is given), on which
its outputs are allocated too; work that made its inputs on another stream has
to be ordered before it, and they have to live until it is done.
"""

from __future__ import annotations

import torch

from . import binding as _b

_DTYPES = {torch.bfloat16: _b.THD_BF16, torch.float16: _b.THD_FP16, torch.float32: _b.THD_FP32}
_F32, _I64, _I32, _U8 = torch.float32, torch.int64, torch.int32, torch.uint8


def _rows_of(logits, name="logits"):
    if logits.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {logits.dtype}")
    if logits.dim() != 2:
        if logits.dim() < 2:
            raise ValueError(f"{name} must be [rows, vocab]")
        try:
            logits = logits.view(-1, logits.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: the leading dimensions cannot be flattened without a copy") from None
    if not logits.is_contiguous():
        if logits.shape[1] > 1 and logits.stride(1) != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        if logits.shape[0] > 1 and logits.stride(0) < logits.shape[1]:
            raise ValueError(f"{name}: rows must not overlap")
    if logits.shape[1] < 1:
        raise ValueError(f"{name} needs at least one column")
    return logits


def _stride(x) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _address(x, name, dtype, count, device, required=False):
    """Address of a contiguous tensor after the checks the C ABI cannot make."""
    if x is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if x.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if x.numel() != count:
        raise ValueError(f"{name} must have {count} elements, got {x.numel()}")
    if x.get_device() != device:
        raise ValueError(f"{name} must be on {f'cuda:{device}' if device >= 0 else 'cpu'}, got {x.device}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


def _need_gpu(x, name):
    if not x.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if x.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {x.device}, which is not the current device")


def _run(call, stream):
    """``call`` with the handle of the stream to use.  Outputs and workspaces are
    allocated inside, on that stream: memory handed back to another stream's
    pool could be given out again too early."""
    if stream is None:
        return call(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


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
    if logits.is_contiguous() and logits.data_ptr() % 16 == 0:
        return torch.empty_like(logits)
    rows, vocab = logits.shape
    size = logits.element_size()
    lead = logits.data_ptr() % 16 // size
    pad = (_stride(logits) - vocab) % (16 // size)
    room = torch.empty(lead + rows * (vocab + pad), dtype=logits.dtype, device=logits.device)
    return room.as_strided((rows, vocab), (vocab + pad, 1), lead)


def _workspace(nbytes, device):
    """(tensor that keeps it alive, address)"""
    if nbytes <= 0:
        return None, None
    room = torch.empty(nbytes, dtype=_U8, device=device)
    return room, room.data_ptr()


def _hand_back(grad, x, out):
    """The gradient in the logits' own shape, or ``out``, written through its
    address: autograd is told, so that an operation which kept ``out`` for its
    own backward reports that it has changed, as for any in-place operation."""
    if out is not None:
        torch.autograd.graph.increment_version(out)
        return out
    return grad if x.dim() == 2 else grad.unflatten(0, x.shape[:-1])


def token_logprobs(logits, labels, mask=None, stream=None):
    """Log-probability of each row's label and the row's log-sum-exp:
    (logp float32 [rows], lse float32 [rows], status)."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    on = z.get_device()
    labels_at = _address(labels, "labels", _I64, rows, on, True)
    mask_at = _address(mask, "mask", _U8, rows, on)
    _need_gpu(z, "logits")
    dtype = _DTYPES[z.dtype]
    lib = _b.library()

    def call(handle):
        dev = z.device
        logp = torch.empty(rows, dtype=_F32, device=dev)
        lse = torch.empty(rows, dtype=_F32, device=dev)
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_loss_workspace_bytes(rows, vocab, dtype, 0)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_token_logprobs(z.data_ptr(), dtype, rows, vocab, _stride(z), labels_at, mask_at,
                                      logp.data_ptr(), lse.data_ptr(), status.data_ptr(), room_at, nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_token_logprobs")
        return logp, lse, status
    return _run(call, stream)


def token_logprobs_backward(dlogp, logits, labels, lse, mask=None, out=None, stream=None):
    """Gradient of ``(dlogp * logp).sum()`` with respect to the logits, in their
    dtype.  ``lse`` is what ``token_logprobs`` returned; ``out`` may be the
    logits themselves, which are then replaced."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    on = z.get_device()
    dlogp_at = _address(dlogp, "dlogp", _F32, rows, on, True)
    labels_at = _address(labels, "labels", _I64, rows, on, True)
    lse_at = _address(lse, "lse", _F32, rows, on, True)
    mask_at = _address(mask, "mask", _U8, rows, on)
    _need_gpu(z, "logits")

    def call(handle):
        grad = _grad_rows(z, out)
        code = _b.library().thd_token_logprobs_backward(
            dlogp_at, z.data_ptr(), _DTYPES[z.dtype], rows, vocab, _stride(z), labels_at, lse_at, mask_at,
            grad.data_ptr(), _stride(grad), handle)
        if code < 0:
            raise _b.ThdError(code, "thd_token_logprobs_backward")
        return _hand_back(grad, logits, out)
    return _run(call, stream)


def policy_loss(logits, labels, old_logp, advantages, mask=None, ref_logp=None, weights=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, out=None, stream=None):
    """Clipped policy loss with a KL term: (loss float32 [rows], logp float32
    [rows], dlogits, status).  ``loss`` holds each row's weighted term (its sum
    is the loss), ``dlogits`` the gradient of that sum; ``weights`` carries the
    normalisation, e.g. one over the number of labelled tokens."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    on = z.get_device()
    labels_at = _address(labels, "labels", _I64, rows, on, True)
    old_at = _address(old_logp, "old_logp", _F32, rows, on, True)
    adv_at = _address(advantages, "advantages", _F32, rows, on, True)
    mask_at = _address(mask, "mask", _U8, rows, on)
    ref_at = _address(ref_logp, "ref_logp", _F32, rows, on)
    weights_at = _address(weights, "weights", _F32, rows, on)
    if kl_coef and ref_logp is None:
        raise ValueError("a KL term needs ref_logp")
    _need_gpu(z, "logits")
    dtype = _DTYPES[z.dtype]
    lib = _b.library()

    def call(handle):
        dev = z.device
        grad = _grad_rows(z, out)
        loss = torch.empty(rows, dtype=_F32, device=dev)
        logp = torch.empty(rows, dtype=_F32, device=dev)
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_loss_workspace_bytes(rows, vocab, dtype, 1)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_policy_loss(z.data_ptr(), dtype, rows, vocab, _stride(z), labels_at, mask_at, old_at, ref_at,
                                   adv_at, weights_at, clip_low, clip_high, kl_coef, loss.data_ptr(),
                                   logp.data_ptr(), grad.data_ptr(), _stride(grad), status.data_ptr(), room_at,
                                   nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_policy_loss")
        return loss, logp, _hand_back(grad, logits, out), status
    return _run(call, stream)


def distill_topk(logits, teacher_logits, teacher_ids, mask=None, weights=None, temperature=1.0, out=None,
                 stream=None):
    """Distillation from a teacher's top logits: (loss float32 [rows], dlogits,
    status).  ``teacher_logits`` [rows, k] and ``teacher_ids`` [rows, k] (int32
    or int64; -1 leaves an entry out) are the teacher's largest logits and their
    columns."""
    z = _rows_of(logits)
    rows, vocab = z.shape
    on = z.get_device()
    if teacher_logits is None or teacher_ids is None:
        raise ValueError("teacher_logits and teacher_ids are required")
    if teacher_ids.dtype not in (_I32, _I64):
        raise ValueError(f"teacher_ids must be int32 or int64, got {teacher_ids.dtype}")
    t = _rows_of(teacher_logits, "teacher_logits")
    k = t.shape[1]
    if k > _b.THD_MAX_TOPK:
        raise ValueError(f"at most {_b.THD_MAX_TOPK} teacher columns, got {k}")
    for name, x in (("teacher_logits", t), ("teacher_ids", teacher_ids)):
        if x.numel() != rows * k or x.shape[-1] != k:
            raise ValueError(f"{name} must be [{rows}, {k}]")
    teacher_at = _address(t, "teacher_logits", t.dtype, rows * k, on)
    ids_at = _address(teacher_ids, "teacher_ids", teacher_ids.dtype, rows * k, on)
    mask_at = _address(mask, "mask", _U8, rows, on)
    weights_at = _address(weights, "weights", _F32, rows, on)
    _need_gpu(z, "logits")
    dtype = _DTYPES[z.dtype]
    lib = _b.library()

    def call(handle):
        dev = z.device
        grad = _grad_rows(z, out)
        loss = torch.empty(rows, dtype=_F32, device=dev)
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_loss_workspace_bytes(rows, vocab, dtype, k)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_distill_topk(z.data_ptr(), dtype, rows, vocab, _stride(z), teacher_at, _DTYPES[t.dtype],
                                    ids_at, teacher_ids.element_size(), k, k, mask_at, weights_at, temperature,
                                    loss.data_ptr(), grad.data_ptr(), _stride(grad), status.data_ptr(), room_at,
                                    nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_distill_topk")
        return loss, _hand_back(grad, logits, out), status
    return _run(call, stream)


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
    on = logp.get_device()
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [pairs, 2]")
    n_pairs = pairs.shape[0]
    if n_pairs > _b.THD_MAX_PAIRS:
        raise ValueError(f"at most {_b.THD_MAX_PAIRS} pairs, got {n_pairs}")
    n_slots = cu_seqlens_padded.numel() - 1
    if n_slots < 0:
        raise ValueError("cu_seqlens_padded needs at least one boundary")
    logp_at = _address(logp, "logp", _F32, total, on)
    ref_at = _address(ref_logp, "ref_logp", _F32, total, on)
    mask_at = _address(mask, "mask", _U8, total, on)
    cu_at = _address(cu_seqlens_padded, "cu_seqlens_padded", _I32, n_slots + 1, on)
    pairs_at = _address(pairs, "pairs", _I32, 2 * n_pairs, on)
    _need_gpu(logp, "logp")
    lib = _b.library()

    def call(handle):
        dev = logp.device
        loss = torch.empty(n_pairs, dtype=_F32, device=dev)
        rewards = torch.empty((n_pairs, 2), dtype=_F32, device=dev)
        dlogp = torch.empty(total, dtype=_F32, device=dev)
        status = torch.empty(1, dtype=_I32, device=dev)
        nbytes = lib.thd_preference_workspace_bytes(total, n_slots)
        room, room_at = _workspace(nbytes, dev)
        code = lib.thd_preference_loss(logp_at, ref_at, mask_at, cu_at, n_slots, total, pairs_at, n_pairs, beta,
                                       label_smoothing, scale, loss.data_ptr(), rewards.data_ptr(),
                                       dlogp.data_ptr(), status.data_ptr(), room_at, nbytes, handle)
        if code < 0:
            raise _b.ThdError(code, "thd_preference_loss")
        return loss, rewards, dlogp, status
    return _run(call, stream)
