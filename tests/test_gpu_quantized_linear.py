"""The example's quantized weights stand for the float ones within half a step of their
grid, also where a group's weights all have one sign."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lo,hi", [(-1.0, 1.0), (1.0, 2.0), (-2.0, -1.0), (0.5, 0.5)])
def test_codes_stand_for_the_weights(lo, hi):
    from attention_layer import QuantizedLinear
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = lo + (hi - lo) * torch.rand(64, 256, generator=g, device="cuda")
    layer = QuantizedLinear(w)
    # the grid spans the group's weights and zero in 15 steps; half a step of rounding, the
    # ends half a step more by the rounded zero, and 2^-11 of the range by the fp16 scale
    step = (max(hi, 0.0) - min(lo, 0.0)) / 15
    assert float((layer.weight - w).abs().max()) <= step * (1 + 15 * 2.0 ** -11)
    x = torch.eye(256, device="cuda").half()
    y = layer(x).float().T
    assert float((y - layer.weight).abs().max()) <= 2.0 ** -9 * float(layer.weight.abs().max())
