"""The example layer runs the block-scaled operators and the balance loss
together, forward and backward, against fp32 torch.

Tolerance: an e4m3 code is off by a uniform error of at most 2^-4 of the value
(2^-4 / sqrt 3 = 3.6 % rms, less for most values), independent from element to
element, so a product of two quantised operands is off by at most sqrt(2) x 3.6
= 5.1 % in the 2-norm and each further quantised step adds 3.6 to 5.1 % (in
squares): two products, the square and its gradient stay below 12 %.  The loss
and the logits' gradient are fp32 throughout.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=3, hidden=256, inner=144, experts=8, k=2, masked=False),
                                   dict(tokens=777, hidden=400, inner=272, experts=24, k=4, seed=3)])
def test_the_layer_matches_fp32(sizes):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from tiled_tensor_core_persistent_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("moe_fp8_layer", os.path.join(HERE, "examples", "moe_fp8_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off = example.run(**sizes)
    for name in ("y", "dx", "dW1", "dW2"):
        assert off[name] < 0.12, off
    assert off["loss"] < 1e-5 and off["dlogits"] < 1e-4, off
