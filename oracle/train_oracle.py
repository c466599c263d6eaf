"""Attention inside documents, the embedding table and the gradients' norm in
NumPy, 64 bits throughout, one document, head or token at a time.

Each function takes arrays on the host and returns float64 arrays of the shapes
the library returns.  Pads are skipped before anything of theirs is read.
"""

from __future__ import annotations

import numpy as np


def share_rows(cu_padded, cu_real, cp, rank):
    """[(row of the share, document's first token, position, document's tokens)] of
    every row of a rank's zigzag share that holds a token (cp 1: of the stream)."""
    cu_padded = [int(c) for c in cu_padded]
    cu_real = cu_padded if cu_real is None else [int(c) for c in cu_real]
    out, row = [], 0
    for s in range(len(cu_padded) - 1):
        start, length = cu_padded[s], cu_padded[s + 1] - cu_padded[s]
        real = cu_real[s + 1] - cu_real[s]
        if cp == 1:
            positions = list(range(length))
        else:
            c = length // (2 * cp)
            positions = [*range(rank * c, (rank + 1) * c), *range((2 * cp - 1 - rank) * c, (2 * cp - rank) * c)]
        for p in positions:
            if p < real:
                out.append((row, start, p, real))
            row += 1
    return out


def visible(i, real, causal, window):
    """Positions that position i of a document of `real` tokens sees."""
    j = np.arange(real)
    keep = np.ones(real, dtype=bool)
    if causal:
        keep &= j <= i
    if window:
        keep &= np.abs(i - j) < window
    return j[keep]


def attention(q, k, v, cu_padded, cu_real=None, causal=True, window=0, scale=None, cap=0.0, cp=1, rank=0):
    """(out [rows, heads, dim], lse [heads, rows])"""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    scale = 1.0 / np.sqrt(dim) if scale is None else scale
    out = np.zeros((rows, heads, dim))
    lse = np.full((heads, rows), -np.inf)
    for row, start, i, real in share_rows(cu_padded, cu_real, cp, rank):
        seen = start + visible(i, real, causal, window)
        for h in range(heads):
            z = scale * (k[seen, h // group].astype(np.float64) @ q[row, h].astype(np.float64))
            if cap:
                z = cap * np.tanh(z / cap)
            top = z.max()
            p = np.exp(z - top)
            out[row, h] = p @ v[seen, h // group].astype(np.float64) / p.sum()
            lse[h, row] = top + np.log(p.sum())
    return out, lse


def attention_backward(dout, q, k, v, cu_padded, cu_real=None, causal=True, window=0, scale=None, cap=0.0, cp=1,
                       rank=0):
    """(dq, dk, dv): gradients of sum(dout * out)."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    scale = 1.0 / np.sqrt(dim) if scale is None else scale
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for row, start, i, real in share_rows(cu_padded, cu_real, cp, rank):
        seen = start + visible(i, real, causal, window)
        for h in range(heads):
            g = h // group
            ks, vs = k[seen, g].astype(np.float64), v[seen, g].astype(np.float64)
            x, d = q[row, h].astype(np.float64), dout[row, h].astype(np.float64)
            z = scale * (ks @ x)
            slope = np.ones_like(z)
            if cap:
                t = np.tanh(z / cap)
                z, slope = cap * t, 1.0 - t * t
            p = np.exp(z - z.max())
            p /= p.sum()
            dp = vs @ d
            dz = p * (dp - p @ dp) * slope * scale
            dq[row, h] = dz @ ks
            dk[seen, g] += np.outer(dz, x)
            dv[seen, g] += np.outer(p, d)
    return dq, dk, dv


def _token_ok(token, vocab):
    return 0 <= int(token) < vocab


def embedding(ids, table, mask=None, scale=1.0):
    out = np.zeros((len(ids), table.shape[1]))
    for t, token in enumerate(ids):
        if mask is None or mask[t]:
            out[t] = scale * table[token].astype(np.float64) if _token_ok(token, len(table)) else np.nan
    return out


def embedding_backward(drows, ids, vocab, mask=None, scale=1.0):
    out = np.zeros((vocab, drows.shape[1]))
    for t, token in enumerate(ids):
        if (mask is None or mask[t]) and _token_ok(token, vocab):
            out[token] += scale * drows[t].astype(np.float64)
    return out


def gradient_norm(grads, scale=1.0):
    return abs(scale) * np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))


def clip_gradients(grads, max_norm, scale=1.0, norm=None):
    """(norm, the scaled gradients); zeros where the norm is not finite in 32 bits."""
    with np.errstate(over="ignore"):
        norm = gradient_norm(grads, scale) if norm is None else norm
        if not np.isfinite(np.float32(norm)):
            return norm, [np.zeros(g.shape) for g in grads]
    factor = scale * min(1.0, max_norm / (norm + 1e-6))
    return norm, [g.astype(np.float64) * factor for g in grads]
