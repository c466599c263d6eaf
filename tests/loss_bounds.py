"""How far a gradient of the losses may be off, column by column.

u = 2^-24 is the half step of 32 bits.  With q the softmax of a row, d the factor
it enters with and [target] the columns the loss names:

    g_v = [target] (what the loss adds) - d q_v

* q_v has the error of its sum and of its exponent, relative to itself:
  (vocab/256 + 280) u + (5 |z_v - max| / tau + 6) u;
* d has an absolute error of its own (from the log-probability, through the
  ratio and the KL term).  It reaches a column times q_v, and only a target's
  column as it is;
* a target's column is one more difference: 8 u |d|;
* the result is rounded once to its type: half a step relative to it, half the
  smallest step of fp16; and the exponential gives 0 below 2^-126.
"""

import numpy as np

U = 2.0 ** -24
# half a step relative to the value, and half the smallest step
HALF = {"bf16": (2.0 ** -8, 0.0), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (U, 0.0)}


def sum_error(vocab):
    return (vocab / 256 + 280) * U


def softmax(z, tau=1.0):
    x = z / tau
    q = np.exp(x - x.max(1, keepdims=True))
    return q / q.sum(1, keepdims=True)


def named(vocab, columns):
    """[row, vocab]: the columns a row's targets name; others than columns name none."""
    out = np.zeros((len(columns), vocab), dtype=bool)
    for t, ids in enumerate(columns):
        ids = np.atleast_1d(ids)
        out[t, ids[(ids >= 0) & (ids < vocab)]] = True
    return out


def gradient_bound(z, d, d_error, grad, target, dtype, tau=1.0, top=None, relative=None):
    """Bound of each element of ``grad``: rows z, factor d of the softmax and its
    error, the columns named as targets.  ``top`` and ``relative`` replace the row's
    maximum and the sum's error where the softmax is taken against a given value."""
    vocab = z.shape[1]
    base = z.max(1, keepdims=True) if top is None else np.asarray(top)[:, None]
    q = softmax(z, tau)
    d, d_error = np.abs(d)[:, None], np.asarray(d_error)[:, None]
    distance = np.abs(z - base) / tau
    rel = (sum_error(vocab) if relative is None else relative) + (5 * np.where(np.isfinite(distance), distance, 0) + 6) * U
    half, tiny = HALF[dtype]
    err = d * (q * rel + 8 * U * target) + d_error * (q + target)
    return err + half * (np.abs(grad) + err) + tiny + 2.0 ** -126 * (1 + d)
