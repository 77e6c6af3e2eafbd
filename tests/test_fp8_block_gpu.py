"""The block norms and the fp8 linears together (examples/fp8_block.py)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_block.py")


@pytest.mark.parametrize("rows,width,heads,samples", [(256, 512, 8, 2), (2, 256, 4, 2), (66, 640, 5, 3)])
def test_block(ops, rows, width, heads, samples):
    spec = importlib.util.spec_from_file_location("fp8_block", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    block = example.Block(width, heads)
    h, mod = example.inputs(rows, width, samples)
    y = block.forward(h, mod, samples)
    ref = block.forward_float(h, mod, samples)
    assert ops.convrot_device_status() == ops.OK
    # A code is off by at most 2^-4 of its value, uniformly: 2^-4 / sqrt 3 of the
    # norm of either operand, 0.051 of a linear's result for both; two linears
    # follow each other on both branches, each branch enters the residual with a
    # gate of 0.3, and its own share of the result's norm is below one half.
    assert float((y.float() - ref).norm() / ref.norm()) < 2 * 2 * 0.051 * 0.5
    # the branches do count: without them the result is far off
    assert float((h.float() - ref).norm() / ref.norm()) > 0.15
    again = block.forward(h, mod, samples)
    assert torch.equal(y, again)
