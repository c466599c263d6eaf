"""The losses on packed streams in NumPy, 64 bits throughout, row by row.

Each function takes arrays on the host and returns float64 arrays of the shapes
the library returns.  Masked rows are skipped before anything of theirs is read.
"""

from __future__ import annotations

import numpy as np


def _rows(mask, n):
    return [t for t in range(n) if mask is None or mask[t]]


def _log_softmax(z):
    """ln softmax of one row; columns at -inf get -inf.  A row with no finite
    maximum has no softmax: NaN."""
    z = np.asarray(z, dtype=np.float64)
    top = z.max()
    if not np.isfinite(top) or np.isnan(z).any():
        return np.full(z.shape, np.nan), np.nan
    lse = top + np.log(np.exp(z - top).sum())
    return (z - top) - np.log(np.exp(z - top).sum()), lse


def _label_ok(y, vocab):
    return 0 <= int(y) < vocab


def token_logprobs(logits, labels, mask=None):
    n, vocab = logits.shape
    logp, lse = np.zeros(n), np.zeros(n)
    for t in _rows(mask, n):
        if not _label_ok(labels[t], vocab):
            logp[t] = lse[t] = np.nan
            continue
        ln_q, lse[t] = _log_softmax(logits[t])
        logp[t] = ln_q[labels[t]]
    return logp, lse


def token_logprobs_backward(dlogp, logits, labels, lse, mask=None):
    n, vocab = logits.shape
    grad = np.zeros((n, vocab))
    for t in _rows(mask, n):
        if not _label_ok(labels[t], vocab):
            grad[t] = np.nan
            continue
        grad[t] = -float(dlogp[t]) * np.exp(np.asarray(logits[t], dtype=np.float64) - float(lse[t]))
        grad[t, labels[t]] += float(dlogp[t])
    return grad


def policy_terms(logp, old, adv, ref, w, clip_low, clip_high, kl_coef):
    """(loss, d loss / d logp) of one row."""
    r = np.exp(logp - old)
    free = r * adv
    held = min(max(r, 1.0 - clip_low), 1.0 + clip_high) * adv
    loss, d = -min(free, held), (-free if free <= held else 0.0)
    if kl_coef:
        u = ref - logp
        loss += kl_coef * (np.expm1(u) - u)
        d -= kl_coef * np.expm1(u)
    return w * loss, w * d


def policy_loss(logits, labels, old_logp, advantages, mask=None, ref_logp=None, weights=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0):
    n, vocab = logits.shape
    loss, logp, grad = np.zeros(n), np.zeros(n), np.zeros((n, vocab))
    for t in _rows(mask, n):
        if not _label_ok(labels[t], vocab):
            loss[t] = logp[t] = np.nan
            grad[t] = np.nan
            continue
        ln_q, _ = _log_softmax(logits[t])
        logp[t] = ln_q[labels[t]]
        loss[t], d = policy_terms(logp[t], float(old_logp[t]), float(advantages[t]),
                                  0.0 if ref_logp is None else float(ref_logp[t]),
                                  1.0 if weights is None else float(weights[t]), clip_low, clip_high, kl_coef)
        grad[t] = -d * np.exp(ln_q)
        grad[t, labels[t]] += d
    return loss, logp, grad


def distill_topk(logits, teacher_logits, teacher_ids, mask=None, weights=None, temperature=1.0):
    n, vocab = logits.shape
    loss, grad = np.zeros(n), np.zeros((n, vocab))
    tau = float(temperature)
    for t in _rows(mask, n):
        ids = [int(i) for i in teacher_ids[t]]
        if any(i < -1 or i >= vocab for i in ids):
            loss[t], grad[t] = np.nan, np.nan
            continue
        part = [(i, float(x)) for i, x in zip(ids, teacher_logits[t]) if i >= 0 and x != -np.inf]
        if not part:
            continue
        w = 1.0 if weights is None else float(weights[t])
        ln_p, _ = _log_softmax(np.array([x for _, x in part]) / tau)
        ln_q, _ = _log_softmax(np.asarray(logits[t], dtype=np.float64) / tau)
        grad[t] = tau * w * np.exp(ln_q)
        for (i, _), lp in zip(part, ln_p):
            p = np.exp(lp)
            grad[t, i] -= tau * w * p
            if p > 0.0:
                loss[t] += tau * tau * w * p * (lp - ln_q[i])
    return loss, grad


def preference_loss(logp, ref_logp, pairs, cu_seqlens_padded, mask=None, beta=0.1, label_smoothing=0.0, scale=1.0):
    logp = np.asarray(logp, dtype=np.float64)
    on = np.ones(len(logp), dtype=bool) if mask is None else np.asarray(mask) != 0
    gap = np.where(on, logp if ref_logp is None else logp - np.asarray(ref_logp, dtype=np.float64), 0.0)
    cu = [int(c) for c in cu_seqlens_padded]
    n_slots = len(cu) - 1
    loss, rewards, dlogp = np.zeros(len(pairs)), np.zeros((len(pairs), 2)), np.zeros(len(logp))
    for i, (c, r) in enumerate(pairs):
        c, r = int(c), int(r)
        if c == -1 and r == -1:
            continue
        if not (0 <= c < n_slots and 0 <= r < n_slots):
            loss[i], rewards[i] = np.nan, np.nan
            continue
        won, lost = slice(cu[c], cu[c + 1]), slice(cu[r], cu[r + 1])
        rewards[i] = beta * gap[won].sum(), beta * gap[lost].sum()
        z = rewards[i, 0] - rewards[i, 1]
        e = label_smoothing
        loss[i] = scale * ((1 - e) * np.logaddexp(0.0, -z) + e * np.logaddexp(0.0, z))
        slope = scale * beta * (e / (1 + np.exp(-z)) - (1 - e) / (1 + np.exp(z)))
        dlogp[won] += slope * on[won]
        dlogp[lost] -= slope * on[lost]
    return loss, rewards, dlogp
