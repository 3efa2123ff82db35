"""The experts' feed-forward example: its stages are the operators' (bit for bit), and the whole is the
64-bit layer up to the quantising.

e4m3 keeps 3 fraction bits: a value is off by at most 2^-4 of itself, 0.4 of that in the mean square, so
each of the four quantised operands (x, two weights, the gated values) adds about 2.6% to the output in
the norm, independently 5.2% together; 10% is asked for."""
import os
import sys

import pytest
import torch

import convolution_onnx_conv_gb300 as cf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,width,hidden,top", [(1, 8, 256, 128, 2), (37, 5, 272, 144, 3), (700, 16, 1024, 768, 2)])
def test_example(tokens, experts, width, hidden, top):
    from expert_feed_forward import example
    y, ref, layer, (x, expert, weight) = example(tokens, experts, width, hidden, top, seed=tokens)
    assert layer.up.status() == cf.CONVF_OK and layer.down.status() == cf.CONVF_OK
    assert float((y - ref).norm() / ref.norm()) < 0.10
    assert torch.equal(layer(x, expert, weight), y)
    # a token by itself gives the row that it gives among the others, up to the order of float32 sums
    one = layer(x[-1:], expert[-1:], weight[-1:])
    assert float((one - y[-1:]).norm() / y[-1:].norm()) < 2.0 ** -6
