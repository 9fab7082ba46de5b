"""GPU tests of the activation and its gradient at gates whose sigmoid is below fp32's normal
numbers, 2^-126 (-87.3 and below), while e^-z still is an fp32 number (to -88.7): silu of them is a
normal number of bf16. Blocks of nothing else, so that these values decide codes and scales. Bounds as in
test_gpu_act, and one more step for the sigmoid: between 2^-128 and 2^-126 it has 22 bits
or more, so it is off by at most 2^-23 of itself more (2 u).
"""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_act import U, backward, bits, check_quantized, forward, inputs
from test_gpu_grouped import dev

import oracle

pytestmark = pytest.mark.gpu


def gates(R, F, act, seed):
    """bf16 gates of -87.5, -88 and -88.5, and others of ordinary size."""
    z, da = inputs(R, F, act, torch.bfloat16, seed)
    z[:, :F] = -87.5 - 0.5 * torch.randint(0, 3, (R, F), generator=torch.Generator().manual_seed(seed))
    return z, da


@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("out", ["e4m3fn", "e5m2", "e2m1"])
@pytest.mark.parametrize("R,F", [(8, 32), (64, 160)])
def test_forward(R, F, out, act):
    progress("act %s %d x %d to %s, far gates" % (act, R, F, out))
    z, _ = gates(R, F, act, R)
    (d, s), _ = mxq.act_quantize(z.cuda(), act, out)
    h, error = forward(z.double().numpy(), F, act)
    assert (h != 0).any()
    check_quantized((d, s), h, error + 2 * U * np.abs(h), z.dtype, out, -1)


@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("out", ["e4m3fn", "e5m2", "e2m1"])
def test_backward(act, out):
    progress("act backward %s to %s, far gates" % (act, out))
    R, F = 64, 160
    z, da = gates(R, F, act, 5)
    z[:, :F] = -88.0                    # a value of e4m3fn
    da = (da * 2.0 ** 10).to(torch.bfloat16)
    d, s = oracle.quantize(bits(z), "bf16", "e4m3fn", layout="dense")
    got = mxq.act_quantize_backward(da.cuda(), dev(d), dev(s), act, "e4m3fn", out)
    kept = oracle.dequantize(d, s, R, z.shape[1], "e4m3fn", layout="dense").astype(np.float64)
    assert (kept[:, :F] == -88.0).all()
    h, herr = forward(kept, F, act)
    dz, derr = backward(da.double().numpy(), kept, F, act)
    check_quantized(got.rows, dz, derr + 4 * U * np.abs(dz), da.dtype, out, -1)
    check_quantized(got.cols, dz, derr + 4 * U * np.abs(dz), da.dtype, out, -2)
    check_quantized(got.h, h, herr + 2 * U * np.abs(h), da.dtype, out, -2)
