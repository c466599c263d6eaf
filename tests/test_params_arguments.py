"""What the Python calls on attention, tables and gradients say about wrong arguments (CPU)."""

import pytest

from context_packed_sequence_amd import params


@pytest.mark.parametrize("bad", [None, 1.5, [1.0]])
def test_gradients_that_are_no_tensors(bad):
    # a parameter without a gradient has None there
    import torch
    g = torch.zeros(4)
    with pytest.raises(ValueError, match=r"grads\[1\] must be a tensor"):
        params._tensors([g, bad, g], "grads", -1)
    with pytest.raises(ValueError, match=r"outs\[0\] must be a tensor"):
        params._tensors([bad], "outs", -1)
