"""Clipping by factors that are no ordinary 32-bit number, on the GPU; tolerances as
counted in test_gpu_params.py."""

import math

import numpy as np
import pytest

import oracle as O
from gpu_util import say
from test_gpu_params import HALF, U, _dtype, _host, _within, thd, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,max_norm,scale", [(1e38, 1e-3, 1.0), (1e36, 1e-6, 1.0), (1e38, 1e-30, -2.0),
                                                 (1e38, math.inf, 1e-42), (1e30, 1e-5, 1.0), (1e-30, 1e-8, 1e30)])
@pytest.mark.parametrize("dtype,out", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")])
def test_small_factors(torch, thd, size, max_norm, scale, dtype, out):
    say("clipping by a small factor", size, max_norm, scale, dtype, out)
    rng = np.random.default_rng(12)
    # below 2^-126 a 32-bit factor has fewer bits, and below 2^-149 none; the products are ordinary numbers
    grads = [torch.from_numpy((rng.uniform(0.1, 1.0, n) * size / 1e3).astype(np.float32)).to(_dtype(torch, dtype)).cuda()
             for n in (20000, 7)]
    host = [_host(g) for g in grads]
    true, want = O.clip_gradients(host, max_norm, scale)
    outs = [torch.empty(g.shape, device="cuda", dtype=_dtype(torch, out)) for g in grads]
    norm, status = thd.clip_gradients(grads, max_norm, scale=scale, outs=outs)
    assert int(status) == 0
    rel = 5 * U + 2 * 20007 * 2.0 ** -53
    for x, y in zip(outs, want):
        half, tiny = HALF[out]
        _within(x, y, (4 * U + rel + half) * np.abs(y) + tiny, "gradient")
    if out == dtype:
        thd.clip_gradients(grads, max_norm, scale=scale)
        assert all(torch.equal(x, y) for x, y in zip(grads, outs))
