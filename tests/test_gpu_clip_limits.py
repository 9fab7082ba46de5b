"""GPU tests of clipping where the factor leaves fp32's normal numbers. Bounds as in
test_gpu_clip: the factor's rounding and the product's, 2^-24 each, and the result
type's."""
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_clip import TYPES, check, rand

pytestmark = pytest.mark.gpu


# a norm of 1e41 clipped to 1 and to less, down to where fp32 has no factor at all,
# and on both sides of 2^-126
@pytest.mark.parametrize("factor", [2.0 ** -125, 2.0 ** -126, 2.0 ** -126 * (1 - 2.0 ** -20), 2.0 ** -127, 1e-41, 1e-44,
                                    1e-46, 1e-60, 1e-100])
@pytest.mark.parametrize("in_place", [False, True])
def test_factors_below_the_normal_numbers(factor, in_place):
    progress("clip by a factor of %g" % factor)
    check([torch.full((1_000_000,), 1e38), rand(777, torch.float32, 3, 1e37), rand(501, torch.bfloat16, 4, 1e37),
           rand(300, torch.float16, 5)], factor, in_place)


@pytest.mark.parametrize("dtype", TYPES)
def test_small_elements_and_a_small_bound(dtype):
    """A factor below 2^-126 on ordinary elements: zeros or the smallest numbers."""
    check([rand(10_001, dtype, 6)], 1e-39)
    check([rand(10_001, dtype, 6, 50.0)], 1e-40)


def test_large_tensors_and_a_tiny_factor():
    """More tiles than the scaling adds the partial sums for by itself."""
    check([torch.full((40_000_003,), 1e38)], 1e-42)


def test_a_tensor_listed_twice_is_refused():
    """In place and as a result; not for the norm, nor without elements."""
    a, b = torch.ones(50, device="cuda"), torch.ones(14, device="cuda")
    with pytest.raises(ValueError):
        mxq.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(ValueError):
        mxq.clip_grad_norm([b, b.clone()], 1.0, out=[b, b])
    assert bool((a == 1).all()) and bool((b == 1).all())
    norm = mxq.grad_norm([a, b, a, a[:14]]).cpu()
    assert torch.equal(norm, torch.tensor(128.0 ** 0.5))     # rounded to fp32
    e = torch.zeros(0, device="cuda")
    assert mxq.clip_grad_norm([a, e, b, e], 4.0).item() == 8.0
    assert bool((a == 0.5).all()) and bool((b == 0.5).all())
