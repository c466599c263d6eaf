"""The oracle of attention, embedding and clipping against differences, closed
forms and itself over other layouts (CPU)."""

import numpy as np
import pytest

import oracle as O
import workloads as W

STEP = 1e-5
CLOSE = dict(rtol=0, atol=1e-8)     # truncation ~ STEP^2, cancellation ~ eps / STEP


def _differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + STEP
        up = f()
        x[i] = keep - STEP
        g[i] = (up - f()) / (2 * STEP)
        x[i] = keep
    return g


def _batch(rng, lens, real, heads=2, kv_heads=1, dim=4, cp=1):
    cu, cu_real = W.cumulative(lens), W.cumulative(real)
    t = int(cu[-1])
    return (rng.normal(size=(t // cp, heads, dim)), rng.normal(size=(t, kv_heads, dim)),
            rng.normal(size=(t, kv_heads, dim)), cu, cu_real)


@pytest.mark.parametrize("how", [dict(), dict(causal=False), dict(window=2), dict(causal=False, window=3),
                                 dict(cap=0.7), dict(cp=2, rank=0), dict(cp=2, rank=1, cap=1.5), dict(scale=0.3)])
def test_attention_gradient_by_differences(how):
    rng = np.random.default_rng(1)
    q, k, v, cu, cu_real = _batch(rng, [8, 0, 4], [5, 0, 4], cp=how.get("cp", 1))
    dout = rng.normal(size=q.shape)

    def loss():
        return float((dout * O.attention(q, k, v, cu, cu_real, **how)[0]).sum())
    got = O.attention_backward(dout, q, k, v, cu, cu_real, **how)
    for name, x, g in zip("qkv", (q, k, v), got):
        np.testing.assert_allclose(g, _differences(loss, x), **CLOSE, err_msg=name)


def test_attention_ranks_make_the_stream():
    # every rank's rows, put where the zigzag layout has them, are the whole stream's
    rng = np.random.default_rng(2)
    cp, lens, real = 4, [16, 8, 24], [13, 8, 1]
    q, k, v, cu, cu_real = _batch(rng, lens, real)
    whole, _ = O.attention(q, k, v, cu, cu_real)
    dout = rng.normal(size=q.shape)
    dq, dk, dv = O.attention_backward(dout, q, k, v, cu, cu_real)
    rows = O.build_route(cu.tolist(), cp, int(cu[-1]))["zigzag"].reshape(cp, -1)  # tokens of each rank's rows
    sum_k, sum_v = 0, 0
    for rank in range(cp):
        at = rows[rank]
        out, _ = O.attention(q[at], k, v, cu, cu_real, cp=cp, rank=rank)
        np.testing.assert_allclose(out, whole[at], rtol=0, atol=1e-12)
        a, b, c = O.attention_backward(dout[at], q[at], k, v, cu, cu_real, cp=cp, rank=rank)
        np.testing.assert_allclose(a, dq[at], rtol=0, atol=1e-12)
        sum_k, sum_v = sum_k + b, sum_v + c
    np.testing.assert_allclose(sum_k, dk, rtol=0, atol=1e-12)
    np.testing.assert_allclose(sum_v, dv, rtol=0, atol=1e-12)


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    q, k, v, cu, _ = _batch(rng, [5, 3], [5, 3], heads=2, kv_heads=2)
    # equal scores: the mean of what is seen
    out, lse = O.attention(q, np.zeros_like(k), v, cu)
    np.testing.assert_allclose(out[6], v[5:7].mean(0), rtol=0, atol=1e-12)
    np.testing.assert_allclose(lse[:, 6], np.log(2), rtol=0, atol=1e-12)
    # a window of one sees itself alone
    np.testing.assert_allclose(O.attention(q, k, v, cu, window=1)[0], v, rtol=0, atol=1e-12)
    # a cap far above the scores changes nothing but their third order
    np.testing.assert_allclose(O.attention(q, k, v, cu, cap=1e4)[0], O.attention(q, k, v, cu)[0], rtol=0, atol=1e-6)


def test_embedding_gradient_is_the_transpose():
    rng = np.random.default_rng(4)
    ids, mask = rng.integers(0, 7, 40), (rng.random(40) < 0.8).astype(np.uint8)
    table, d = rng.normal(size=(7, 5)), rng.normal(size=(40, 5))
    lhs = float((d * O.embedding(ids, table, mask, 0.5)).sum())
    rhs = float((O.embedding_backward(d, ids, 7, mask, 0.5) * table).sum())
    assert abs(lhs - rhs) < 1e-12
    ids[3], mask[3] = 7, 1
    assert np.isnan(O.embedding(ids, table, mask)[3]).all()
    assert np.isfinite(O.embedding_backward(d, ids, 7, mask)).all()


def test_clipped_norm():
    rng = np.random.default_rng(5)
    grads = [rng.normal(size=n) for n in (1, 0, 17)]
    norm, out = O.clip_gradients(grads, 0.5, scale=2.0)
    assert abs(O.gradient_norm(out) - 0.5 * norm / (norm + 1e-6)) < 1e-12
    norm, out = O.clip_gradients(grads, 1e9, scale=2.0)
    np.testing.assert_allclose(out[2], 2 * grads[2])
    grads[2][4] = np.nan
    assert not any(o.any() for o in O.clip_gradients(grads, 1.0)[1])


@pytest.mark.parametrize("how", [dict(), dict(causal=False, window=3), dict(cap=0.7), dict(cp=2, rank=1)])
def test_bounds_hold_the_oracle_values(how):
    # the bounds' own values are the oracle's, and a mistake of a few roundings' size is outside
    import attention_bounds
    rng = np.random.default_rng(6)
    q, k, v, cu, cu_real = _batch(rng, [12, 4], [9, 4], heads=4, kv_heads=2, dim=8, cp=how.get("cp", 1))
    dout = rng.normal(size=q.shape)
    got = attention_bounds.attention("bf16", q, k, v, cu, cu_real, dout=dout, **how)
    out, lse = O.attention(q, k, v, cu, cu_real, **how)
    want = dict(zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *O.attention_backward(dout, q, k, v, cu, cu_real, **how))))
    for name, (value, bound) in got.items():
        np.testing.assert_allclose(value, want[name], rtol=0, atol=1e-12, err_msg=name)
        assert (bound[np.isfinite(value)] <= 0.2 * np.abs(value[np.isfinite(value)]).max()).all(), name
