"""The microscaled operators together, as examples/mx_layer.py uses them."""
import os
import sys

import pytest
import torch

from parity import gpu_lib

pytestmark = pytest.mark.gpu


def test_example_trains_and_its_two_forward_paths_agree():
    gpu_lib()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import mx_layer
    first, last, y4, y = mx_layer.train(steps=40, log=lambda s: None)
    assert last < 0.5 * first
    # The same 4-bit codes and products, quantised ahead or on the way.
    assert torch.equal(y4, y)
