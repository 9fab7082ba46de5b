"""GPU tests of the layer for a few tokens on weights at the ends of their formats: codes
with the smallest scale bytes, which are below what bf16 holds, and e5m2's infinities. Bounds
as in test_gpu_few_tokens.
"""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_few_tokens import STEP, case, check, reference
from test_gpu_grouped import host

pytestmark = pytest.mark.gpu


def subnormal(codes, fmt, seed):
    """Every code a subnormal of the format (e2m1: its smallest two), zeros among them."""
    g = np.random.default_rng(seed)
    if fmt == "e2m1":
        n = g.integers(0, 3, (2, *codes.shape)) | g.integers(0, 2, (2, *codes.shape)) << 3
        codes[:] = n[0] | n[1] << 4
    else:
        codes[:] = g.integers(0, 8 if fmt == "e4m3fn" else 4, codes.shape) | g.integers(0, 2, codes.shape) << 7


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3fn", "e5m2"])
@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("T,k,E,K,F,N", [(6, 2, 3, 96, 32, 36), (40, 2, 2, 544, 64, 68)])
def test_smallest_scales(T, k, E, K, F, N, act, fmt):
    """Scale bytes 0 .. 12 in every block of the first weights, then of the second, and
    activations that bring the results back to ordinary sizes: all of a result comes from such
    weights."""
    def up(x, w1, w2):
        g = np.random.default_rng(3)
        subnormal(w1[0], fmt, 4)
        w1[1][:] = g.integers(0, 13, w1[1].shape)
        x[:] = x * 2.0 ** (120 if fmt != "e2m1" else 110)

    check(*case(T, k, E, K, F, N, fmt, act, torch.bfloat16, patch=up))

    def down(x, w1, w2):
        g = np.random.default_rng(5)
        subnormal(w2[0], fmt, 6)
        w2[1][:] = g.integers(0, 13, w2[1].shape)
        w1[1][:, :, F:] += 110          # the other's columns: the gates stay ordinary

    if act == "swiglu":
        check(*case(T, k, E, K, F, N, fmt, act, torch.bfloat16, patch=down))


@pytest.mark.parametrize("fmt,low", [("e4m3fn", 1), ("e5m2", 8)])
def test_smallest_scales_of_f16_rows(fmt, low):
    """(h is about 2^-112, and the second weights' scales of 2^100 and more bring it back.)"""
    def patch(x, w1, w2):
        subnormal(w1[0], fmt, 4)
        w1[1][:] = np.random.default_rng(3).integers(low, low + 2, w1[1].shape)
        x[:] = x * 2.0 ** 13
        w2[1][:] = w2[1] + 110

    check(*case(9, 2, 3, 544, 64, 68, fmt, "silu", torch.float16, patch=patch))


def test_smallest_scales_beside_ordinary_ones():
    """A block of zeros with a small scale byte, as a quantized zero has, and blocks of one
    column that need not be another's."""
    def patch(x, w1, w2):
        w1[0][:, :8, :] = 0
        w1[1][:, 0, :] = 1
        w2[1][:, 0, ::3] = 2

    for fmt in ("e4m3fn", "e5m2"):
        check(*case(20, 2, 3, 96, 64, 36, fmt, "swiglu", torch.bfloat16, patch=patch))
        check(*case(20, 2, 3, 96, 64, 36, fmt, "silu", torch.float16, patch=patch))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("which", ["first", "second"])
def test_infinite_weights(which, act, dtype):
    progress("few tokens, an infinity in the %s weights, %s %s" % (which, act, dtype))

    def patch(x, w1, w2):
        q, s = w1 if which == "first" else w2
        q[1, 5, 4 * 7 + 2] = 0x7C           # expert 1: row 22 of column 7
        q[1, 1, 4 * 9 + 1] = 0xFC
        s[1, 0, 9] = 255

    with np.errstate(all="ignore"):
        call, plain = case(9, 2, 4, 96, 64, 68, "e5m2", act, dtype, patch=patch)
        want, bound = reference(*plain)
    got = host(mxq.moe_few_tokens(*call))
    top = 65504.0 if dtype == torch.float16 else 3.3895313892515355e38
    assert (np.abs(want[np.isfinite(want)]) < top).all()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    fin = np.isfinite(want)
    assert fin.any() and not fin.all()
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    got, want, bound = got[fin], want[fin], bound[fin]
    assert (np.abs(got - want) <= bound + STEP[dtype] * (np.abs(want) + bound) + tiny).all()
