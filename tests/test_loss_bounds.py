"""The gradient bound of the GPU tests tells a right gradient from a wrong one (CPU)."""

import numpy as np
import pytest

import oracle as O
from loss_bounds import U, gradient_bound, named, sum_error


def _round(g, dtype):
    torch = pytest.importorskip("torch")
    return torch.from_numpy(g).to({"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]).double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [1000, 32000, 131075])
def test_blocks_off_the_label_are_checked(dtype, vocab):
    rng = np.random.default_rng([3, vocab])
    n = 3
    z = rng.normal(0, 3, (n, vocab))
    labels = np.array([0, vocab // 2, vocab - 1])
    z[np.arange(n), labels] += 4
    logp, _ = O.token_logprobs(z, labels)
    old, adv, w = logp - 0.1, np.array([0.7, -1.3, 0.4]), np.array([1.0, 0.3, 0.6])
    _, _, grad = O.policy_loss(z, labels, old, adv, weights=w)
    d = -adv * w * np.exp(logp - old)
    e_logp = sum_error(vocab) + 4 * U * 20
    bound = gradient_bound(z, d, np.abs(d) * (e_logp + 8 * U), grad, named(vocab, labels), dtype)

    def off(got):
        return np.abs(got - grad) > bound
    assert not off(_round(grad, dtype)).any()
    for at in (8, vocab // 3 // 8 * 8, vocab - 24):
        block = np.setdiff1d(np.arange(at, at + 8), labels)
        zeroed, shifted, scaled = grad.copy(), grad.copy(), grad.copy()
        zeroed[:, block] = 0
        shifted[:, block] = grad[:, block + 8 if at + 16 < vocab else block - 8]
        scaled[:, block] *= 1.02 if dtype == "bf16" else 1.001
        for wrong in (zeroed, shifted, scaled):
            assert off(_round(wrong, dtype))[:, block].mean() > 0.9
    # the label's own term, left out or given to a neighbour
    for t in range(n):
        wrong = grad.copy()
        wrong[t, labels[t]] = -d[t] * np.exp(z[t, labels[t]] - z[t].max()) / np.exp(z[t] - z[t].max()).sum()
        assert off(_round(wrong, dtype))[t, labels[t]]
