"""The activations between products, the products with 4-bit weights and the layer for a
few tokens run together, as examples/gated_moe.py has them.

e4m3 with block scales is off by at most 2^-4 of a value, spread evenly: at most
2^-4 / sqrt(3) = 3.6 % in the norm, each operand by itself. A training step's result has
six such roundings in it (x and W1, in the gate and its partner, h and W2): 3.6 % sqrt(6) =
8.9 %. A gradient has up to twelve (those of z, and z's 8 bits, in both factors; dy, dh's W2,
dz, and the other operand): 12.5 %. With the served weights' own values a prompt has three
(x in both, h): 6.2 %, and a decode step rounds nothing but the result, by 2^-8 of it at
most. A wrong row, expert, weight or layout is off by 100 %.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

SIZES = [(1000, 2, 8, 512, 1024), (37, 4, 32, 256, 96), (3000, 3, 4, 320, 544), (1, 1, 2, 32, 32)]


@pytest.mark.parametrize("tokens,slots,experts,K,F", SIZES[:3])
def test_training_step(tokens, slots, experts, K, F):
    import gated_moe

    for name, d in gated_moe.train(tokens, slots, experts, K, F).items():
        assert d < 0.15, (name, d)


@pytest.mark.parametrize("tokens,slots,experts,K,F", SIZES)
def test_serving(tokens, slots, experts, K, F):
    import gated_moe

    prompt, decode = gated_moe.serve(tokens, slots, experts, K, F)
    assert prompt < 0.1, prompt
    assert decode < 2.0 ** -8, decode


def test_decode_graph():
    import gated_moe

    assert gated_moe.decode_graph()
