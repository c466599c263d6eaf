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


def test_the_device_named():
    # neither attention nor the table has logits to compare with
    import torch

    from context_packed_sequence_amd.losses import _address
    with pytest.raises(ValueError, match="ids must be on cuda:1, got cpu"):
        _address(torch.zeros(4, dtype=torch.int64), "ids", torch.int64, 4, 1)
