"""The mixture-of-experts calls run together, as examples/moe_step.py has them.

e4m3 with block scales rounds each operand by up to 2^-4 of its value (about
2^-5 on average), so one product of two such operands is about 2^-5 sqrt(2) =
4 % off in the norm, and a chain of two (the layer, or a gradient through it)
twice that at most; a wrong row, expert, weight or layout is off by 100 %.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,slots,experts,K,F", [(1000, 2, 8, 512, 1024), (37, 4, 32, 256, 96), (1, 1, 2, 32, 32),
                                                      (3000, 3, 4, 320, 544)])
def test_training_step(tokens, slots, experts, K, F):
    import moe_step

    distance, before, after = moe_step.step(tokens, slots, experts, K, F, max_norm=0.5)
    for name, d in distance.items():
        assert d < 0.12, (name, d)
    assert before > 0.5 and abs(after - 0.5) < 0.5 * 2.0 ** -8


def test_decode_graph():
    import moe_step

    assert moe_step.decode_graph()
