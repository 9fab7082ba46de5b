"""GPU tests of e5m2's infinities (codes 0x7C and 0xFC, as torch's conversion to float8_e5m2
writes where a value is too large) in the FP8 products, on either side and beside scale bytes
of 255: results are those of the sums in 64 bits. Bounds as in test_gpu_grouped.
"""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_fp4_infinities import MINUS, PLUS, compare
from test_gpu_grouped import dev, host, quantized, values

pytestmark = pytest.mark.gpu


def place(codes, C, spots):
    """Infinities at (k, column, code) of a [K, C] operand."""
    at = codes.reshape(-1, C, 4)
    for k, c, code in spots:
        at[k // 4, c, k % 4] = code


def scales(ls, rs, where):
    """Bytes of 255 (2^128) on one side, small ones opposite."""
    if where in ("left", "both"):
        ls[0, ::3], rs[..., 0, :] = 255, 20
    if where in ("right", "both"):
        rs[..., -1, 1::3], ls[-1, :] = 255, 20


def operand(K, C, dim, seed, K_last):
    q, s = quantized(C if dim == -1 else K, K if dim == -1 else C, dim, "e5m2", seed)
    place(q, C, [(1, C - 1, PLUS), (K_last, 0, MINUS), (2, C // 2, PLUS), (K_last - 1, C // 2, MINUS)])
    return q, s


@pytest.mark.parametrize("where", ["nowhere", "left", "right", "both"])
@pytest.mark.parametrize("M,K,N", [(4, 32, 4), (72, 160, 136), (516, 96, 260), (260, 288, 516)])
def test_product(M, K, N, where):
    progress("FP8 product with infinities %d x %d x %d, 255: %s" % (M, K, N, where))
    l, ls = operand(K, M, -1, M, K - 1)
    r, rs = operand(K, N, -2, N + 1, K - 3)
    scales(ls, rs, where)
    for res in (torch.float32, torch.bfloat16):
        got = host(mxq.scaled_matmul(dev(l), dev(ls), dev(r), dev(rs), "e5m2", res, dense_scale=True))
        want = compare(got, values(l, ls, "e5m2"), values(r, rs, "e5m2"), res)
        assert np.isinf(want).any()


# streamed, 128-row and 256-row tiles
@pytest.mark.parametrize("where", ["nowhere", "left", "right", "both"])
@pytest.mark.parametrize("sizes,K,N", [([32, 0, 8], 96, 132), ([128, 160, 132], 160, 516), ([700, 132, 516], 672, 516)])
def test_groups(sizes, K, N, where):
    progress("FP8 groups with infinities %s, %d x %d, 255: %s" % (sizes, K, N, where))
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = int(offsets[-1])
    l, ls = operand(K, rows, -1, rows, K - 1)
    r, rs = (np.stack(t) for t in zip(*[operand(K, N, -2, N + g, K - 3) for g in range(len(sizes))]))
    scales(ls, rs, where)
    got = host(mxq.grouped_scaled_matmul(dev(l), dev(ls), dev(r), dev(rs), dev(offsets), "e5m2", torch.float32))
    L = values(l, ls, "e5m2")
    for g, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if a != b:
            compare(got[a:b], L[:, a:b], values(r[g], rs[g], "e5m2"), torch.float32)


@pytest.mark.parametrize("where", ["nowhere", "left", "right", "both"])
def test_wgrad(where):
    sizes, M, N = [64, 0, 96, 32], 132, 68
    progress("weight gradients with infinities, 255: %s" % where)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = int(offsets[-1])
    l, ls = operand(rows, M, -2, 5, rows - 1)
    r, rs = operand(rows, N, -2, 6, rows - 3)
    scales(ls, rs, where)
    got = host(mxq.grouped_scaled_matmul_wgrad(dev(l), dev(ls), dev(r), dev(rs), dev(offsets), "e5m2", torch.float32))
    L, R = values(l, ls, "e5m2"), values(r, rs, "e5m2")
    for g, (a, b) in enumerate(zip(offsets, offsets[1:])):
        if a != b:
            compare(got[g], L[a:b], R[a:b], torch.float32)


def test_what_torch_writes():
    """torch's conversion gives an infinity where a value is past the largest one."""
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn((64, 96), generator=g), torch.randn((96, 32), generator=g)
    x[3, 40] = 1e6
    code = lambda a: a.to(torch.float8_e5m2).view(torch.uint8)      # noqa: E731
    l = code(x).view(64, 24, 4).permute(1, 0, 2).reshape(24, 256).contiguous()
    r = code(w).view(24, 4, 32).permute(0, 2, 1).reshape(24, 128).contiguous()
    ones = [torch.full((3, c), 127, dtype=torch.uint8) for c in (64, 32)]
    got = host(mxq.scaled_matmul(l.cuda(), ones[0].cuda(), r.cuda(), ones[1].cuda(), "e5m2", torch.float32,
                                 dense_scale=True))
    want = compare(got, values(l.numpy(), ones[0].numpy(), "e5m2"), values(r.numpy(), ones[1].numpy(), "e5m2"),
                   torch.float32)
    assert np.isinf(want[3]).sum() > 24
