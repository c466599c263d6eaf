"""Values at the ends of their range: rows without a softmax, references without
probability, extreme temperatures, and gradients in place of saved logits."""

import numpy as np
import pytest

import oracle as O
from gpu_util import say
from test_gpu_losses import (  # noqa: F401  (the fixtures torch and thd)
    U, Case, _check_distill, _check_matrix, _host, _logp_error, _sum_error, _within, thd, torch)

pytestmark = pytest.mark.gpu

# one workgroup per row, few rows in parts, rows of a wide workgroup
SHAPES = [(1100, 3001), (5, 70001), (300, 20000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_rows_without_a_softmax_stay_nan(torch, thd, rows, vocab, dtype):
    # the log-sum-exp of nothing but -inf is NaN like that of +inf and NaN, and
    # so is the gradient made from it
    say("no softmax", dtype, rows, vocab)
    case = Case(torch, 40, 5, rows, vocab, dtype)
    z, labels, d = case.logits, case.dev(case.labels), case.dev(case.d)
    z[1::5] = -float("inf")
    z[2::5, vocab // 3] = float("inf")
    z[3::5, vocab - 1] = float("nan")
    logp, lse, status = thd.token_logprobs(z, labels)
    assert int(status.item()) == 0
    grad = thd.token_logprobs_backward(d, z, labels, lse)
    for i in (1, 2, 3):
        assert bool(torch.isnan(logp[i::5]).all()) and bool(torch.isnan(lse[i::5]).all())
        assert bool(torch.isnan(grad[i::5].float()).all())
    for i in (0, 4):
        assert bool(torch.isfinite(lse[i::5]).all()) and bool(torch.isfinite(grad[i::5].float()).all())


@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_reference_without_probability(torch, thd, rows, vocab):
    # u = ref - logp towards -inf: exp(u) - 1 goes to -1 however large the loss
    say("reference", rows, vocab)
    case = Case(torch, 41, 5, rows, vocab, "fp32")
    case.mask[:] = 1
    kl = 0.3
    logp, _ = O.token_logprobs(case.z, case.labels)
    case.ref = np.array([-np.inf, -3e38, -1e9, logp[3] - 40, logp[4] - 0.6], dtype=np.float32)
    loss, got, grad, _ = thd.policy_loss(
        case.logits, case.dev(case.labels), case.dev(case.old), case.dev(case.adv), ref_logp=case.dev(case.ref),
        weights=case.dev(case.w), clip_low=0.2, clip_high=0.3, kl_coef=kl)
    want = O.policy_loss(case.z, case.labels, case.old, case.adv, None, case.ref, case.w, 0.2, 0.3, kl)
    assert np.isinf(want[0][0]) and np.isfinite(want[2]).all()
    e_logp, _ = _logp_error(case.z, case.labels)
    _within(_host(got), case.whole(want[1]), case.whole(e_logp), "logp")
    r = np.exp(want[1] - case.old)
    e_ratio = np.abs(case.adv) * r * (e_logp + (np.abs(want[1] - case.old) * 4 + 6) * U)
    u = case.ref.astype(np.float64) - want[1]
    with np.errstate(invalid="ignore"):
        e_exp = np.where(u < -300, 0.0, np.exp(u) * (e_logp + (6 + 4 * np.abs(u)) * U))
    e_d = case.w * (e_ratio + kl * (e_exp + 2 * U)) + 6 * U * case.w * (np.abs(case.adv) * r + kl)
    e_loss = case.w * (e_ratio + 4 * U * 1.3 * np.abs(case.adv) + kl * (e_exp + e_logp)) + 8 * U * np.abs(want[0])
    _within(_host(loss), case.whole(want[0]), case.whole(e_loss), "loss")
    d = np.array([O.loss_oracle.policy_terms(want[1][t], case.old[t], case.adv[t], case.ref[t], case.w[t], 0.2, 0.3,
                                             kl)[1] for t in range(5)])
    z = case.z
    soft = np.exp(z - z.max(1, keepdims=True))
    soft /= soft.sum(1, keepdims=True)
    label = np.arange(vocab) == case.labels[:, None]
    rel = _sum_error(vocab) + (5 * np.abs(z - z.max(1, keepdims=True)) + 6) * U
    bound = np.abs(d)[:, None] * (soft * rel + 8 * U * label) + e_d[:, None] * (soft + label) + U * np.abs(want[2])
    _check_matrix(case, grad, want[2], bound + 2.0 ** -126, "gradient")


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("tau,weight", [(2.0 ** -80, 2.0 ** 60), (2.0 ** 80, 2.0 ** -100)])
def test_temperatures_whose_square_leaves_32_bits(torch, thd, rows, vocab, tau, weight):
    # tau^2 itself is 2^-160 or 2^160; tau^2 w (ln p - ln q) is an ordinary number
    say("temperature", rows, vocab, tau)
    case = Case(torch, 42, 5, rows, vocab, "fp32", k=4)
    case.mask[:] = 1
    if tau < 1:
        # far below any distance of two logits: p and q are the largest's alone
        case.ids[:, 0] = case.z.argmin(1)
        case.teacher[:, 0] = 9
    case.w[:] = weight
    loss, _, status = thd.distill_topk(case.logits, case.dev(case.teacher).contiguous(),
                                       case.dev(case.ids).contiguous(), weights=case.dev(case.w), temperature=tau)
    assert int(status.item()) == 0
    want, _ = O.distill_topk(case.z, case.teacher.astype(np.float64), case.ids, None, case.w, tau)
    assert (want > 2.0 ** -30).all() and (want < 2.0 ** 100).all()
    # a sum of k terms, ln q of size ln V or |z - max| / tau, the sum behind it
    _within(_host(loss), case.whole(want), case.whole((_sum_error(vocab) + 40 * U) * np.abs(want)), "loss")


def test_gradient_in_place_of_saved_logits(torch, thd):
    # an operation that keeps its result for its own backward notices that the
    # gradient has replaced it
    say("in place and autograd")
    x = torch.randn((12, 500), device="cuda", requires_grad=True)
    y = torch.zeros(12, dtype=torch.int64, device="cuda")
    f = torch.zeros(12, device="cuda")
    t, ids = torch.zeros((12, 2), device="cuda"), torch.zeros((12, 2), dtype=torch.int32, device="cuda")
    for call in (lambda z: thd.policy_loss(z, y, f, f + 1, out=z)[2],
                 lambda z: thd.distill_topk(z, t, ids, out=z)[1],
                 lambda z: thd.token_logprobs_backward(f + 1, z, y, f + 7, out=z)):
        capped = 30 * torch.tanh(x / 30)          # the product keeps nothing of its result
        capped.backward(call(capped.detach()))
        kept = torch.tanh(x)                      # its backward needs the result
        grad = call(kept.detach())
        assert grad.data_ptr() == kept.data_ptr()
        with pytest.raises(RuntimeError, match="inplace operation"):
            kept.backward(grad)
    with torch.inference_mode():
        z = torch.randn((12, 500), device="cuda")
        assert thd.policy_loss(z, y, f, f + 1, out=z)[2] is z
