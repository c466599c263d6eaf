"""The losses of few long rows, each cut into parts over several workgroups.

Rows take that form from 8193 16-byte words on for log-probabilities (up to 64
rows) and from 4097 on for the losses (up to 48 rows).  Oracle, cases and bounds
are those of test_gpu_losses.
"""

import numpy as np
import pytest

from gpu_util import say
from test_gpu_losses import (  # noqa: F401  (the fixtures torch and thd)
    Case, _check_distill, _dtype, thd, torch)

pytestmark = pytest.mark.gpu


def _in_parts(thd, case, targets):
    kind = {"bf16": thd.THD_BF16, "fp16": thd.THD_FP16, "fp32": thd.THD_FP32}[case.dtype]
    return thd.thd_loss_workspace_bytes(case.rows, case.vocab, kind, targets) > 0


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("dtype,vocab,stride,offset", [
    ("fp32", 33003, 33003, 0), ("bf16", 50257, 50264, 0), ("fp16", 50257, 50257, 5), ("bf16", 131075, 131075, 0)])
def test_teacher_columns_at_both_ends(torch, thd, rows, dtype, vocab, stride, offset):
    # a gradient at another place than the logits: the elements before the first
    # and after the last whole word have one owner, targets or not
    say("ends of the row", rows, dtype, vocab)
    case = Case(torch, 31, 3, rows, vocab, dtype, stride=stride, offset=offset, k=20)
    assert _in_parts(thd, case, 20)
    case.mask[:] = 1
    case.ids[:, :8] = np.arange(8)
    case.ids[:, 8:16] = vocab - 1 - np.arange(8)
    case.ids[1, 16:] = vocab - 1                # the last column several times
    case.ids[2, 1:19] = -1                      # and hardly anything else
    case.ids[2, 19] = vocab - 1
    for _ in range(3):
        _check_distill(case, thd, out="elsewhere", tau=1.5, teacher_dtype=_dtype(torch, dtype))
    _check_distill(case, thd, out="in place", tau=1.5)
