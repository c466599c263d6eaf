"""How tight the attention's bounds are (CPU): a mistake of a few half steps of the
largest value is outside, at every element."""

import numpy as np
import pytest

import attention_bounds
from test_train_oracle import _batch

# half steps of the result's type (32 bits for lse).  out: p's rounding and its own, each at most
# the largest value's; dv the same with rows in p's place; dq and dk: dz's rounding, delta's from
# the rounded out and their own, with terms that cancel in the value but not in the bound
STEPS = {"out": 3, "lse": 48, "dq": 16, "dk": 16, "dv": 4}


@pytest.mark.parametrize("how", [dict(), dict(causal=False, window=3), dict(cap=0.7), dict(cp=2, rank=1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_few_half_steps_are_outside(how, dtype):
    rng = np.random.default_rng(6)
    q, k, v, cu, cu_real = _batch(rng, [12, 4], [9, 4], heads=4, kv_heads=2, dim=8, cp=how.get("cp", 1))
    got = attention_bounds.attention(dtype, q, k, v, cu, cu_real, dout=rng.normal(size=q.shape), **how)
    assert set(got) == set(STEPS)
    for name, (value, bound) in got.items():
        live = np.isfinite(value)
        half = 2.0 ** -24 if name == "lse" else attention_bounds.HALF[dtype]
        assert (bound[live] < STEPS[name] * half * np.abs(value[live]).max()).all(), name
