"""GPU tests of the products where a wave's part of a tile lies past the result's last
row or column while the operands hold scale bytes of 255 or NaN codes: such a part
takes no second pass and changes no result. Bounds as in test_gpu_grouped."""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_grouped import check_rows, compare, dev, host, quantized, values
from test_gpu_grouped_forms import check_wgrad

pytestmark = pytest.mark.gpu


def scales(l, ls, r, rs):
    """255 in the last block's last columns, small scales on the other side."""
    ls[-1, -3:] = 255
    ls[-1, :-3] = 100
    rs[..., -1, -1] = 255
    rs[..., -1, :-1] = 24


def codes(l, ls, r, rs):
    l[-1, -1] = 0x7F
    r[..., -1, -4] = 0xFF


# widths whose last 256-column tile has less than 128 columns, and rows whose last
# tile has 64 or less; 4 by 4: the operand is shorter than a wave's start column
@pytest.mark.parametrize("patch", [scales, codes])
@pytest.mark.parametrize("sizes,M,N", [([32, 64], 4, 4), ([64], 4, 300), ([32, 0, 64], 260, 4), ([800], 300, 260),
                                       ([1536], 4, 4)])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_wgrad(sizes, M, N, res, patch):
    progress("grouped wgrad %s M=%d N=%d %s %s" % (sizes, M, N, res, patch.__name__))
    check_wgrad(sizes, M, N, "e4m3fn", res, 41, patch, per_block=4)


@pytest.mark.parametrize("patch", [scales, codes])
@pytest.mark.parametrize("sizes,K,N", [([132, 68, 260], 96, 2564), ([500, 700, 604], 96, 2600),
                                       ([500, 700, 604], 1056, 2600), ([32] * 3, 64, 4)])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_rows(sizes, K, N, res, patch):
    progress("grouped rows %s K=%d N=%d %s %s" % (sizes, K, N, res, patch.__name__))
    check_rows(sizes, 0, K, N, "e4m3fn", res, seed=43, patch=patch, per_block=4)


@pytest.mark.parametrize("patch", [scales, codes])
@pytest.mark.parametrize("M,N", [(4, 4), (300, 260), (4, 300), (516, 292)])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_scaled_matmul(M, N, res, patch):
    progress("scaled matmul M=%d N=%d %s %s" % (M, N, res, patch.__name__))
    l, ls = quantized(160, M, -2, "e4m3fn", M)
    r, rs = quantized(160, N, -2, "e4m3fn", N + 1)
    patch(l, ls, r, rs)
    big = torch.full((M * N + 64,), 7.0, dtype=res, device="cuda")
    mxq.scaled_matmul(dev(l), dev(ls), dev(r), dev(rs), "e4m3fn", res, out=big[:M * N].view(M, N), dense_scale=True)
    got = host(big)
    assert (got[M * N:] == 7).all()
    compare(got[:M * N].reshape(M, N), values(l, ls, "e4m3fn"), values(r, rs, "e4m3fn"), res, 4)


@pytest.mark.parametrize("first,sizes,tail", [(4, [32], 0), (64, [32, 0, 64], 0), (36, [40, 8], 12), (128, [0, 0], 0),
                                              (700, [132, 68, 260], 40), (96, [32] * 80, 4)])
@pytest.mark.parametrize("K,N", [(64, 36), (96, 2600), (1056, 132)])
def test_rows_before_the_first_group(first, sizes, tail, K, N):
    """Offsets of some experts of a plan: the rows before them are zeros, like those
    past them, and nothing is written beyond either."""
    progress("grouped rows, %d before the first group, %s, %d past" % (first, sizes, tail))
    offsets = (first + np.concatenate([[0], np.cumsum(sizes)])).astype(np.int32)
    rows, G = int(offsets[-1]) + tail, len(sizes)
    l, ls = quantized(rows, K, -1, "e4m3fn", rows)
    r, rs = (np.stack(t) for t in zip(*[quantized(K, N, -2, "e4m3fn", g % 7) for g in range(G)]))
    big = torch.full((rows * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    mxq.grouped_scaled_matmul(dev(l), dev(ls), dev(r), dev(rs), dev(offsets), "e4m3fn", torch.bfloat16,
                              out=big[:rows * N].view(rows, N))
    got = host(big)
    assert (got[rows * N:] == 7).all()
    got = got[:rows * N].reshape(rows, N)
    assert (got[:first] == 0).all() and (got[offsets[-1]:] == 0).all()
    L = values(l, ls, "e4m3fn")
    for g in range(G):
        a, b = offsets[g], offsets[g + 1]
        if a != b:
            compare(got[a:b], L[:, a:b], values(r[g], rs[g], "e4m3fn"), torch.bfloat16)


def test_part_of_a_plan_by_experts():
    """The products of a plan's experts in two calls, each on its experts' offsets and
    weights, add up to those of one call."""
    g = np.random.default_rng(5)
    E, K, N = 16, 64, 132
    plan = mxq.moe_sort(torch.from_numpy(g.integers(0, E, size=(300, 2))).cuda(), E)
    rows = plan.src.numel()
    l, ls = map(dev, quantized(rows, K, -1, "e4m3fn", 1))
    r, rs = (dev(np.stack(t)) for t in zip(*[quantized(K, N, -2, "e4m3fn", e) for e in range(E)]))
    whole = mxq.grouped_scaled_matmul(l, ls, r, rs, plan.offsets)
    parts = [mxq.grouped_scaled_matmul(l, ls, r[a:b], rs[a:b], plan.offsets[a:b + 1]) for a, b in ((0, 8), (8, 16))]
    assert torch.equal(parts[0] + parts[1], whole)
