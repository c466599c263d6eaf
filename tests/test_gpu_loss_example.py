"""The losses together, as examples/packed_losses.py uses them."""

import importlib.util
import math
import os

import pytest

from conftest import ROOT
from gpu_util import say

pytestmark = pytest.mark.gpu


def test_example_learns_from_every_loss():
    say("example: packed losses")
    spec = importlib.util.spec_from_file_location("packed_losses", os.path.join(ROOT, "examples", "packed_losses.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for name, values in example.run(steps=6).items():
        assert all(math.isfinite(v) for v in values), name
        assert values[-1] < values[0], (name, values)
