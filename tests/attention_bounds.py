"""How far the attention's results may be off, element by element.

u = 2^-24 is the half step of 32 bits, w that of the tensors' type (bf16 2^-8, fp16
2^-11), n a row's keys, D the head's elements.  Scores are sums of D exact products in
32 bits, through a tanh where they are capped (absolute error 6 u of a number up to
1: two instructions good to 2 u each and three roundings) and an exponential
(instruction and argument's rounding):

    e_z   = (D + 4) u scale sum |q k|, + 8 u cap, + 4 u |z|
    r_p   = 2 max e_z + (n + 16) u              relative error of a probability
    lse   : max e_z + (n + 16) u + 4 u |lse|

A probability is rounded to w of itself as a factor (fp16: and by up to 2^-35, half the
smallest step over the power of two it is held with in the backward pass, and by
2^-25 in the forward pass), and a result once to its type:

    out   : (w + r_p + n u) sum p |v| + w |out|
    dv    : the same with sums over the rows
    dz    : p (1 - t^2) ((D + 4) u sum |dout v| + (D + 4) u sum |dout out| + sum |dout| e_out),
            where e_out is out's bound: delta is formed from the rounded out;
            + (w + r_p + 16 u) |dz|, + p |dp - delta| 16 u of the slope 1 - t^2 where capped
            (fp16: and by up to 2^-38 of 2 max |dout| max |v|)
            (and see below: numbers under 2^-126)
    dq, dk: sums of |k|, |q| times dz's bound, + n u sum |dz k| + w |dq|

The exponential instruction gives 0 below 2^-126, and products and factors of the
matrix instructions may be taken as 0 there, too: a probability is off by up to F =
2^-126 besides, dz by F (|dp - delta| + 1), and each term of a sum, and the result, by F.
"""

import numpy as np

U = 2.0 ** -24
F = 2.0 ** -126
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25}


def _pieces(cu_padded, cu_real, cp, rank):
    """(rows, document's start, positions, document's tokens) of each document of a share."""
    import oracle as O
    found = {}
    for row, start, p, real in O.share_rows(cu_padded, cu_real, cp, rank):
        found.setdefault(start, ([], [], real))
        found[start][0].append(row)
        found[start][1].append(p)
    return [(np.array(r), s, np.array(p), real) for s, (r, p, real) in found.items()]


def attention(dtype, q, k, v, cu_padded, cu_real=None, causal=True, window=0, scale=None, cap=0.0, cp=1, rank=0,
              dout=None):
    """{name: (value, bound)} of out and lse, and of dq, dk, dv where there is a dout."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    scale = 1.0 / np.sqrt(dim) if scale is None else scale
    w, tiny = HALF[dtype], TINY[dtype]
    narrow = dtype == "fp16"
    val = {"out": np.zeros(q.shape), "lse": np.full((heads, rows), -np.inf), "dq": np.zeros(q.shape),
           "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    err = {n: np.zeros(x.shape) for n, x in val.items()}
    if dout is not None:
        top = 2 * max((np.linalg.norm(dout[r], axis=-1).max(initial=0) for r, _, _, _ in
                       _pieces(cu_padded, cu_real, cp, rank)), default=0)
        top *= max((np.linalg.norm(v[s:s + real], axis=-1).max(initial=0) for _, s, _, real in
                    _pieces(cu_padded, cu_real, cp, rank)), default=0)
    for r, start, pos, real in _pieces(cu_padded, cu_real, cp, rank):
        at = slice(start, start + real)
        i, j = pos[:, None], np.arange(real)[None]
        sees = np.ones((len(pos), real), dtype=bool)
        if causal:
            sees &= j <= i
        if window:
            sees &= np.abs(i - j) < window
        n = sees.sum(1, keepdims=True)
        for h in range(heads):
            g = h // group
            x, ks, vs = q[r, h], k[at, g], v[at, g]
            z = scale * (x @ ks.T)
            e_z = (dim + 4) * U * scale * (np.abs(x) @ np.abs(ks).T)
            slope = np.ones_like(z)
            if cap:
                t = np.tanh(z / cap)
                z, slope = cap * t, 1 - t * t
                e_z = e_z + 8 * U * cap
            e_z = e_z + 4 * U * np.abs(z)
            z = np.where(sees, z, -np.inf)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            total = p.sum(1, keepdims=True)
            p /= total
            worst = np.where(sees, e_z, 0).max(1, keepdims=True)
            r_p = 2 * worst + (n + 16) * U
            val["lse"][h, r] = (m + np.log(total))[:, 0]
            err["lse"][h, r] = (worst + (n + 16) * U)[:, 0] + 4 * U * np.abs(val["lse"][h, r])
            o = p @ vs
            e_o = (w + r_p + n * U) * (p @ np.abs(vs)) + w * np.abs(o) + tiny + F * (sees @ (np.abs(vs) + 1) + 1)
            if narrow:
                e_o = e_o + 2.0 ** -25 * (sees @ np.abs(vs))
            val["out"][r, h], err["out"][r, h] = o, e_o
            if dout is None:
                continue
            d = dout[r, h]
            dp = d @ vs.T
            delta = (d * o).sum(1, keepdims=True)
            dz = p * (dp - delta) * slope
            e_dz = p * slope * ((dim + 4) * U * (np.abs(d) @ np.abs(vs).T + (np.abs(d) * np.abs(o)).sum(1, keepdims=True))
                                + (np.abs(d) * e_o).sum(1, keepdims=True))
            e_dz = e_dz + (w + r_p + 16 * U) * np.abs(dz) + 16 * U * p * np.abs(dp - delta) * (cap > 0)
            e_dz = e_dz + F * (np.abs(dp - delta) + 1) * sees
            if narrow:
                e_dz = e_dz + top * 2.0 ** -38 * sees
            val["dq"][r, h] = scale * (dz @ ks)
            err["dq"][r, h] = scale * ((e_dz + n * U * np.abs(dz)) @ np.abs(ks))
            m_rows = sees.sum(0)[:, None] * group
            val["dk"][at, g] += scale * (dz.T @ x)
            err["dk"][at, g] += scale * (e_dz.T @ np.abs(x) + m_rows * U * (np.abs(dz).T @ np.abs(x)))
            val["dv"][at, g] += p.T @ d
            e_p = (w + r_p) * p + F * sees + (2.0 ** -35 * sees if narrow else 0)
            err["dv"][at, g] += e_p.T @ np.abs(d) + m_rows * U * (p.T @ np.abs(d))
    for name in ("dq", "dk", "dv"):
        err[name] += w * np.abs(val[name]) + tiny + F * (rows + k.shape[0])
    names = ["out", "lse"] + (["dq", "dk", "dv"] if dout is not None else [])
    return {name: (val[name], err[name]) for name in names}
