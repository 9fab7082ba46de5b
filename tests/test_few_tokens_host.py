"""The workspace that the layer for a few tokens asks for: no GPU needed."""
import pytest

import mx_microscaling_quantization_amd as mxq


def up16(n):
    return -(-n // 16) * 16


@pytest.mark.parametrize("tokens,slots,F,N", [(1, 1, 0, 4), (1, 1, 32, 4), (1024, 1, 32, 4), (1024, 1, 32, 64), (1024, 1, 32, 68),
                                              (333, 3, 32, 132), (16, 64, 64, 2012), (16, 4, 2048, 4096), (3, 5, 32, 0)])
def test_workspace_holds_every_part(tokens, slots, F, N):
    """h as two planes of 16 bits, y in fp32, and a counter for each token and tile of 64
    columns, each part from a multiple of 16 bytes on."""
    pairs = tokens * slots
    least = up16(4 * pairs * F) + up16(4 * pairs * N) + 4 * -(-N // 64) * tokens
    assert mxq.load().mxq_moe_few_tokens_workspace_bytes(tokens, slots, F, N) >= least


def test_no_tokens_need_none():
    assert mxq.load().mxq_moe_few_tokens_workspace_bytes(0, 2, 32, 64) == 0
