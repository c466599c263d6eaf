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
