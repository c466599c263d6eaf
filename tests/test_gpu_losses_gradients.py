"""Every gradient element against the oracle, with the bound of loss_bounds: what
a row's factor is off by counts at the columns its targets name, elsewhere
only in proportion to the element.  Each form of the kernels, each type, and
gradients in every place a caller can put them."""

import numpy as np
import pytest

import oracle as O
from gpu_util import say
from loss_bounds import U, gradient_bound, named, sum_error
from test_gpu_losses import (  # noqa: F401  (the fixtures torch and thd)
    Case, _check_matrix, _dtype, _logp_error, thd, torch)

pytestmark = pytest.mark.gpu

# rows in parts; one workgroup per row of every size; rows beyond registers and LDS
SHAPES = [(3, 70001), (40, 50257), (3, 163851), (1100, 1000), (1100, 4104), (530, 16390), (530, 32000), (300, 65543),
          (270, 98311), (270, 131075), (60, 230003)]
OUTS = ["new", "in place", "elsewhere", "contiguous"]


def _place(case, kind):
    """A tensor for the gradient: None, the logits, rows at another place within
    16 bytes, or packed rows beside logits whose rows are padded."""
    torch = case.torch
    if kind == "new":
        return None
    if kind == "in place":
        return case.logits
    if kind == "contiguous":
        return torch.empty((case.rows, case.vocab), dtype=case.logits.dtype, device="cuda")
    room = torch.full((case.rows * (case.vocab + 3) + 5,), 7.0, dtype=case.logits.dtype, device="cuda")
    return room.as_strided((case.rows, case.vocab), (case.vocab + 3, 1), 1 + case.offset)


def _case(torch, seed, rows, vocab, dtype, out, k=0):
    n = 3 if vocab > 40000 else 5
    stride = vocab + 16 - vocab % 8 if out == "contiguous" else vocab
    return Case(torch, seed, n, rows, vocab, dtype, stride=stride, k=k)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_policy(torch, thd, rows, vocab, dtype, out):
    say("policy", rows, vocab, dtype, out)
    case = _case(torch, 50, rows, vocab, dtype, out)
    case.labels[:3] = [0, vocab - 1, vocab // 2]      # the row's ends too
    logp, _ = O.token_logprobs(case.z, case.labels)
    case.old = (logp + np.array([0.1, -0.15, 0.05, -0.1, 0.12])[:case.n]).astype(np.float32)
    case.ref = (logp + np.array([0.4, -0.3, 0.1, -0.7, 0.6])[:case.n]).astype(np.float32)
    case.mask[:] = 1
    kl = 0.3
    _, _, grad, _ = thd.policy_loss(
        case.logits, case.dev(case.labels), case.dev(case.old), case.dev(case.adv), ref_logp=case.dev(case.ref),
        weights=case.dev(case.w), clip_low=0.2, clip_high=0.3, kl_coef=kl, out=_place(case, out))
    _, logp, want = O.policy_loss(case.z, case.labels, case.old, case.adv, None, case.ref, case.w, 0.2, 0.3, kl)
    e_logp, _ = _logp_error(case.z, case.labels)
    r, u = np.exp(logp - case.old), case.ref - logp
    e_d = case.w * (np.abs(case.adv) * r * (e_logp + (np.abs(logp - case.old) * 4 + 12) * U)
                    + kl * (np.exp(u) * (e_logp + (12 + 4 * np.abs(u)) * U) + 6 * U))
    d = np.array([O.loss_oracle.policy_terms(logp[t], case.old[t], case.adv[t], case.ref[t], case.w[t], 0.2, 0.3, kl)[1]
                  for t in range(case.n)])
    _check_matrix(case, grad, want,
                  gradient_bound(case.z, d, e_d, want, named(vocab, case.labels), dtype), "gradient")


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_log_probabilities(torch, thd, rows, vocab, dtype, out):
    say("logp backward", rows, vocab, dtype, out)
    case = _case(torch, 51, rows, vocab, dtype, out)
    case.labels[:3] = [0, vocab - 1, vocab // 2]
    _, lse = O.token_logprobs(case.z, case.labels)
    lse = lse.astype(np.float32)
    grad = thd.token_logprobs_backward(case.dev(case.d), case.logits, case.dev(case.labels), case.dev(lse),
                                       out=_place(case, out))
    want = O.token_logprobs_backward(case.d, case.z, case.labels, lse)
    d = case.d.astype(np.float64)
    bound = gradient_bound(case.z, d, 2 * U * np.abs(d), want, named(vocab, case.labels), dtype,
                           top=lse.astype(np.float64), relative=4 * U)
    _check_matrix(case, grad, want, bound, "gradient")


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_distillation(torch, thd, rows, vocab, dtype, out):
    say("distillation", rows, vocab, dtype, out)
    k, tau = 37, 1.5
    case = _case(torch, 52, rows, vocab, dtype, out, k=k)
    case.ids[:, :6] = [0, 1, 2, vocab - 3, vocab - 2, vocab - 1]     # the row's ends too
    case.ids[0, 30:] = -1
    case.ids[1, 20:24] = case.ids[1, 7]                              # a column given five times
    case.mask[:] = 1
    teacher = torch.from_numpy(case.teacher).to(_dtype(torch, dtype))
    _, grad, _ = thd.distill_topk(case.logits, teacher.cuda()[torch.from_numpy(case.pick).cuda()].contiguous(),
                                  case.dev(case.ids).to(torch.int32).contiguous(), weights=case.dev(case.w),
                                  temperature=tau, out=_place(case, out))
    t = teacher.double().numpy()
    _, want = O.distill_topk(case.z, t, case.ids, None, case.w, tau)
    c = tau * case.w.astype(np.float64)
    target = named(vocab, case.ids)
    bound = gradient_bound(case.z, c, 2 * U * c, want, target, dtype, tau=tau)
    # a target's probability: k additions, an argument of size |t - max|, its repeats added up
    spread = t.max(1) - t.min(1)
    bound += target * (c * (2 * k + 20 + 5 * spread / tau) * U)[:, None] * 1.01
    _check_matrix(case, grad, want, bound, "gradient")
