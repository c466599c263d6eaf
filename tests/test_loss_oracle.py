"""The loss oracle against central differences and closed forms (CPU)."""

import math

import numpy as np
import pytest

import oracle as O

STEP = 1e-5
# central differences in 64 bits: truncation ~ STEP^2, cancellation ~ eps / STEP
CLOSE = dict(rtol=0, atol=1e-8)


def _differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + STEP
        up = f(x)
        x[i] = keep - STEP
        down = f(x)
        x[i] = keep
        g[i] = (up - down) / (2 * STEP)
    return g


@pytest.fixture
def rng():
    return np.random.default_rng(5)


def _batch(rng, n=6, vocab=9):
    z = rng.normal(0, 1.5, (n, vocab))
    labels = rng.integers(0, vocab, n)
    mask = np.ones(n, dtype=np.uint8)
    mask[2] = 0
    return z, labels, mask


def test_logprob_gradient(rng):
    z, labels, mask = _batch(rng)
    d = rng.normal(size=len(labels))
    _, lse = O.token_logprobs(z, labels, mask)
    got = O.token_logprobs_backward(d, z, labels, lse, mask)
    want = _differences(lambda x: float((d * O.token_logprobs(x, labels, mask)[0]).sum()), z)
    np.testing.assert_allclose(got, want, **CLOSE)
    assert not got[2].any()


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient(rng, kl):
    z, labels, mask = _batch(rng, n=12)
    now, _ = O.token_logprobs(z, labels)
    # ratios on both sides of both ends, with either sign of the advantage, none within a step of an end
    old = now + np.array([-0.6, -0.3, -0.1, 0.1, 0.3, 0.6] * 2)
    adv = np.repeat([1.3, -0.7], 6)
    ref = now + rng.normal(0, 0.5, 12)
    w = rng.uniform(0.2, 1, 12)

    def run(x):
        return O.policy_loss(x, labels, old, adv, mask, ref, w, 0.2, 0.3, kl)
    want = _differences(lambda x: float(run(x)[0].sum()), z)
    np.testing.assert_allclose(run(z)[2], want, **CLOSE)


@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_distill_gradient(rng, tau):
    z, _, mask = _batch(rng)
    ids = np.array([rng.permutation(9)[:4] for _ in range(6)])
    ids[1, 2] = -1
    ids[3, 3] = ids[3, 0]           # a column given twice
    ids[4] = -1                     # nothing left
    t = rng.normal(0, 2, (6, 4))
    t[5, 1] = -np.inf
    w = rng.uniform(0.2, 1, 6)
    loss, got = O.distill_topk(z, t, ids, mask, w, tau)
    want = _differences(lambda x: float(O.distill_topk(x, t, ids, mask, w, tau)[0].sum()), z)
    np.testing.assert_allclose(got, want, **CLOSE)
    assert loss[4] == 0 and not got[4].any()


def test_preference_gradient(rng):
    cu = [0, 3, 3, 8, 12, 14]
    pairs = [(0, 2), (3, 2), (4, 1), (-1, -1), (0, 0)]
    mask = np.ones(14, dtype=np.uint8)
    mask[[1, 9, 13]] = 0
    logp, ref = rng.normal(-2, 1, 14), rng.normal(-2, 1, 14)

    def run(x):
        return O.preference_loss(x, ref, pairs, cu, mask, 0.7, 0.1, 0.5)
    loss, rewards, got = run(logp)
    want = _differences(lambda x: float(run(x)[0].sum()), logp)
    np.testing.assert_allclose(got, want, **CLOSE)
    assert loss[3] == 0 and not rewards[3].any()
    # a document against itself tells nothing
    assert loss[4] == pytest.approx(0.5 * math.log(2)) and rewards[4, 0] == rewards[4, 1]


def test_closed_forms():
    z = np.full((1, 7), -3.0)
    logp, lse = O.token_logprobs(z, [4])
    assert logp[0] == pytest.approx(-math.log(7)) and lse[0] == pytest.approx(-3 + math.log(7))
    assert O.token_logprobs(np.array([[5.0]]), [0])[0][0] == 0.0
    # a teacher equal to the student over the whole vocabulary: no loss, no gradient
    z = np.array([[0.3, -1.0, 2.0]])
    loss, grad = O.distill_topk(z, z, [[0, 1, 2]], temperature=2.0)
    assert loss[0] == pytest.approx(0) and np.allclose(grad, 0)
    # the same policy as before, at its own reference: the loss is -A, the gradient A (q - [y])
    old, _ = O.token_logprobs(z, [2])
    loss, _, grad = O.policy_loss(z, [2], old, [1.5], ref_logp=old, kl_coef=0.2)
    q = np.exp(z[0]) / np.exp(z[0]).sum()
    assert loss[0] == pytest.approx(-1.5)
    np.testing.assert_allclose(grad[0], 1.5 * (q - np.array([0, 0, 1])), atol=1e-12)


def test_rows_that_leave_nothing():
    z = np.full((2, 3), np.nan)
    loss, logp, grad = O.policy_loss(z, [-5, 99], [0, 0], [1, 1], mask=[0, 0])
    assert not loss.any() and not logp.any() and not grad.any()
    assert np.isnan(O.token_logprobs(np.zeros((1, 3)), [3])[0]).all()
    assert np.isnan(O.token_logprobs(np.full((1, 3), -np.inf), [1])[0]).all()
