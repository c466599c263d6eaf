"""What the loss calls refuse or need at the ends of their range (CPU)."""

import pytest

import context_packed_sequence_amd as thd

# addresses far apart; nothing is read through them
Z, G, MASK, W, LOSS, STATUS, T, ID = (i << 32 for i in range(1, 9))


def _distill(temperature):
    return thd.binding.library().thd_distill_topk(
        Z, thd.THD_BF16, 600, 32000, 32000, T, thd.THD_FP32, ID, 8, 16, 16, MASK, W, temperature, LOSS, G, 32000,
        STATUS, None, 0, None)


@pytest.mark.parametrize("temperature", [3.0e-39, 4.0e-39, 4.2e-39])
def test_temperatures_too_small_for_the_exponent_factor(temperature):
    # 1 / tau is a 32-bit number there, log2(e) / tau is not: every exponent
    # would be a product with infinity
    assert _distill(temperature) == thd.THD_ERR_ARG
