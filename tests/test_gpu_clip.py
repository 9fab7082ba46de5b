"""GPU tests of the global norm and clipping against 64-bit sums.

The squares are added in 64 bits, so the norm is off by its rounding to fp32,
2^-24 (and the sums' own n 2^-53). A scaled element is off by the factor's
rounding, the product's (2^-24 each) and the result type's eps / 2; an f16
result below 2^-14 by at most 2^-25, a result below 2^-126 by 2^-133 (bf16) or
2^-149 (f32).
"""
import math

import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def exact_norm(tensors):
    return math.sqrt(math.fsum(t.double().square().sum().item() for t in tensors))


def check(tensors, factor, in_place=False):
    tensors = [t.cuda() for t in tensors]
    before = [t.clone() for t in tensors]
    norm = exact_norm(before)
    max_norm = factor * norm
    out = None if in_place else [torch.full_like(t, 3.0) for t in tensors]
    got = mxq.clip_grad_norm(tensors, max_norm, out=out)
    assert got.dtype == torch.float32 and got.dim() == 0
    if norm < (2.0 - 2.0 ** -24) * 2.0 ** 127:
        assert abs(got.item() - norm) <= 2.0 ** -23.9 * norm
    else:   # a norm beyond fp32 rounds to infinity; the scaling uses the 64-bit one
        assert got.item() == math.inf
    scale = max_norm / norm if norm > max_norm else 1.0
    for b, t in zip(before, tensors if in_place else out):
        want = b.double() * scale
        if scale == 1.0:
            assert torch.equal(t, b)
        else:
            eps = 0.0 if t.dtype == torch.float32 else torch.finfo(t.dtype).eps / 2
            tol = want.abs() * (2 * 2.0 ** -23.9 + eps * (1 + 2.0 ** -22)) + SMALLEST[t.dtype]
            assert bool(((t.double() - want).abs() <= tol).all())
    if not in_place:
        for b, t in zip(before, tensors):
            assert torch.equal(b, t), "an input changed"
    assert mxq.grad_norm(before).item() == got.item()


def rand(n, dtype, seed, scale=0.02):
    return (torch.randn(n, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 4096, 8191, 8192, 8193, 100003])
def test_one_tensor(n, dtype):
    progress("clip one tensor of %d %s" % (n, dtype))
    check([rand(n, dtype, n)], 0.3)


@pytest.mark.parametrize("factor", [0.0, 0.1, 0.999, 1.5])
@pytest.mark.parametrize("in_place", [False, True])
def test_mixed_tensors(factor, in_place):
    ts = [rand(1 + 977 * i % 30011, TYPES[i % 3], i) for i in range(40)]
    check(ts, factor, in_place)


@pytest.mark.parametrize("count", [112, 113, 300])
def test_more_tensors_than_one_launch(count):
    progress("clip %d tensors" % count)
    ts = [rand(5 + 61 * i % 9001, TYPES[i % 3], i) for i in range(count)]
    check(ts, 0.25)
    check(ts, 0.25, in_place=True)


def test_empty_tensors_and_shapes():
    check([torch.zeros(0), rand((3, 5, 7), torch.float32, 1), torch.zeros((4, 0), dtype=torch.float16),
           rand((1,), torch.bfloat16, 2)], 0.5)
    only = [torch.zeros(0, device="cuda")]
    assert mxq.clip_grad_norm(only, 1.0).item() == 0.0 and mxq.grad_norm(only).item() == 0.0
    z = [torch.zeros(100, device="cuda")]
    assert mxq.clip_grad_norm(z, 0.0).item() == 0.0


def test_values_whose_squares_leave_fp32():
    check([torch.full((1000,), 3e30), rand(77, torch.float32, 3)], 0.5)
    check([torch.full((1000,), 1e-30), torch.full((10,), 2e-38)], 0.5)
    check([torch.full((5000,), 3e38, dtype=torch.bfloat16)], 0.5e-3)
    check([torch.full((33,), 65504.0, dtype=torch.float16), torch.full((5,), 6e-8, dtype=torch.float16)], 0.1)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_changes_nothing(bad):
    for dtype in TYPES:
        t = rand(5001, dtype, 4)
        t[4321] = bad
        t = t.cuda()
        keep, out = t.clone(), torch.zeros_like(t)
        norm = mxq.clip_grad_norm([t], 1e-3, out=[out]).item()
        assert not math.isfinite(norm)
        bits = torch.int32 if dtype == torch.float32 else torch.int16
        assert torch.equal(out.view(bits)[:4321], keep.view(bits)[:4321])
        mxq.clip_grad_norm([t], 1e-3)
        assert torch.equal(t.view(bits), keep.view(bits))


def test_tensors_at_element_alignment():
    """Views that start at any element."""
    base = rand(4000, torch.bfloat16, 5).cuda()
    out = torch.full_like(base, 9.0)
    v, o = base[1:2050], out[3:2052]
    mxq.clip_grad_norm([v, base[2051:2052]], 0.01, out=[o, out[3001:3002]])
    norm = exact_norm([v, base[2051:2052]])
    want = v.double() * (0.01 / norm)
    assert bool(((o.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -21) + 2.0 ** -133).all())
    assert bool((out[:3] == 9).all()) and bool((out[2052:3001] == 9).all()) and bool((out[3002:] == 9).all())


def test_refusals():
    t = torch.zeros((4, 6), device="cuda")
    with pytest.raises(ValueError):
        mxq.clip_grad_norm([t.t()], 1.0)
    with pytest.raises(ValueError):
        mxq.clip_grad_norm([t], 1.0, out=[t[0]])
    with pytest.raises(ValueError):
        mxq.clip_grad_norm([t.double()], 1.0)


def test_stream_graph_and_repeats():
    ts = [rand(1 + 3001 * i, TYPES[i % 3], i).cuda() for i in range(20)]
    out = [torch.empty_like(t) for t in ts]
    want_norm = mxq.clip_grad_norm(ts, 0.5, out=out).clone()
    want = [o.clone() for o in out]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        n = mxq.clip_grad_norm(ts, 0.5, out=out, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(n, want_norm) and all(torch.equal(a, b) for a, b in zip(out, want))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n = mxq.clip_grad_norm(ts, 0.5, out=out)
    for _ in range(4):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, want_norm) and all(torch.equal(a, b) for a, b in zip(out, want))
        _ = ts[3].float().sum().item()


@pytest.mark.parametrize("in_place", [False, True])
def test_large_tensors(in_place):
    """More tiles than the scaling adds the partial sums for by itself (128 MiB),
    alone and with more tensors than one launch holds."""
    big = [torch.randn(50_000_003, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16),
           rand(17_000_001, torch.float32, 2)]
    check(big, 0.3, in_place)
    check(big + [rand(1 + 37 * i, TYPES[i % 3], i) for i in range(130)], 0.3, in_place)
