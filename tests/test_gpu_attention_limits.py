"""Attention at the ends of its scales, against the oracle (64 bits)."""

import pytest

from gpu_util import say
from test_gpu_attention import Batch, _check, thd, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


# scores near 0 from ordinary values, and scores of a few from very large and very small ones
@pytest.mark.parametrize("scale,spread", [(2.0 ** -100, 1.0), (2.0 ** -100, 2.0 ** 48.5), (2.0 ** 100, 2.0 ** -51.5)])
@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_ends_of_the_scales(torch, thd, scale, spread, cap):
    say("attention ends of the scales", scale, spread, cap)
    _check(thd, Batch(torch, [140, 61], [133, 61], heads=2, dim=64, scale=scale, spread=spread, cap=cap), "scales")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("grad", [1.0, 2.0 ** -12])
def test_smallest_cap(torch, thd, dtype, grad):
    # scores that are all the cap or minus it: their slope is 0 but near 0, gradients of scores nothing
    say("attention smallest cap", dtype, grad)
    _check(thd, Batch(torch, [70], heads=2, dim=64, dtype=dtype, cap=2.0 ** -64, grad=grad), "smallest cap")
