"""GPU tests of the experts' products where the number of tiles, the length of the
contraction and the rows per group pick another form, and of what is cleared
without a product. Bounds as in test_gpu_grouped.

rows:  128 x 256 tiles on up to half of the CUs, or up to 64 rows per group: 32-row
       tiles; else up to 384 rows per group or 1024 values: 128-row tiles;
       else 256-row tiles
wgrad: fewer than 768 rows of the contraction per group: 128-row tiles, else 256
"""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_grouped import check_rows, compare, dev, host, quantized, values

pytestmark = pytest.mark.gpu

MANY = [500, 700, 600]      # 15 + 1 tiles of 128 rows; 11 of 256 columns


def scales(l, ls, r, rs):
    ls[1, 3:150] = 255
    rs[:, 1, :] = 20
    rs[:, 0, ::5] = 255
    ls[0, :] = 14


def codes(l, ls, r, rs):
    l[3, 4 * 630 + 2] = 0x7F
    r[1, 2, 4 * 1017 + 1] = 0xFF


@pytest.mark.parametrize("patch", [None, scales, codes])
@pytest.mark.parametrize("fmt,res,N", [("e4m3fn", torch.bfloat16, 2624), ("e4m3fn", torch.float32, 2600)])
def test_short_contraction(fmt, res, N, patch):
    """128-row tiles; N = 2624: rows of results are whole 128-byte lines."""
    progress("grouped rows, 128-row tiles, N=%d %s" % (N, patch))
    check_rows(MANY, 20, 96, N, fmt, res, seed=4, patch=patch, per_block=4)


@pytest.mark.parametrize("sizes", [[200, 0, 384, 380, 500, 260, 364], [300] * 7])
def test_middling_groups_of_many_tiles(sizes):
    progress("grouped rows, 128-row tiles of middling groups %s" % sizes)
    check_rows(sizes, 60, 128, 2052, "e5m2", torch.bfloat16, seed=14)


@pytest.mark.parametrize("patch", [None, scales, codes])
@pytest.mark.parametrize("fmt,res,N", [("e4m3fn", torch.bfloat16, 2624), ("e4m3fn", torch.float32, 2600)])
def test_long_contraction(fmt, res, N, patch):
    """256-row tiles"""
    progress("grouped rows, 256-row tiles, N=%d %s" % (N, patch))
    check_rows(MANY, 20, 1056, N, fmt, res, seed=5, patch=patch, per_block=4)


@pytest.mark.parametrize("sizes", [[1024], [516, 0, 700], [600, 4, 8]])
def test_few_tiles_of_many_rows(sizes):
    """32-row tiles for large groups too: a narrow result has few others."""
    progress("grouped rows, few tiles %s" % sizes)
    check_rows(sizes, 36, 1056, 132, "e4m3fn", torch.bfloat16, seed=6)
    check_rows(sizes, 36, 160, 516, "e5m2", torch.float32, seed=7)


@pytest.mark.parametrize("sizes,N", [([4], 4), ([0, 8], 12), ([32] * 3, 36), ([500, 700, 600], 1156)])
@pytest.mark.parametrize("tail", [4, 36, 1300])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_rows_past_the_last_group(sizes, N, tail, res):
    """Cleared to the last byte, 8 of them past the last 16 among these, and nothing
    beyond."""
    progress("grouped rows, %d past the last group, N=%d" % (tail, N))
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    real, rows, G = int(offsets[-1]), int(offsets[-1]) + tail, len(sizes)
    l, ls = quantized(rows, 32, -1, "e4m3fn", rows)
    r, rs = (np.stack(t) for t in zip(*[quantized(32, N, -2, "e4m3fn", g) for g in range(G)]))
    big = torch.full((rows * N + 64,), 7.0, dtype=res, device="cuda")
    mxq.grouped_scaled_matmul(dev(l), dev(ls), dev(r), dev(rs), dev(offsets), "e4m3fn", res,
                              out=big[:rows * N].view(rows, N))
    got = host(big)
    assert (got[real * N:rows * N] == 0).all() and (got[rows * N:] == 7).all()
    L = values(l, ls, "e4m3fn")
    for g in range(G):
        a, b = offsets[g], offsets[g + 1]
        if a != b:
            compare(got[a * N:b * N].reshape(b - a, N), L[:, a:b], values(r[g], rs[g], "e4m3fn"), res)


def check_wgrad(sizes, M, N, fmt, res, seed, patch=None, per_block=1):
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows, G = int(offsets[-1]), len(sizes)
    l, ls = quantized(rows, M, -2, fmt, seed)
    r, rs = quantized(rows, N, -2, fmt, seed + 1)
    if patch:
        patch(l, ls, r, rs)
    big = torch.full((G * M * N + 64,), 7.0, dtype=res, device="cuda")
    mxq.grouped_scaled_matmul_wgrad(dev(l), dev(ls), dev(r), dev(rs), dev(offsets), fmt, res,
                                    out=big[:G * M * N].view(G, M, N))
    got, L, R = host(big), values(l, ls, fmt), values(r, rs, fmt)
    assert (got[G * M * N:] == 7).all()
    got = got[:G * M * N].reshape(G, M, N)
    for g in range(G):
        a, b = offsets[g], offsets[g + 1]
        if a == b:
            assert (got[g] == 0).all()
        else:
            compare(got[g], L[a:b], R[a:b], res, per_block)


# 768 rows per group on average and one block less
@pytest.mark.parametrize("sizes", [[768], [736], [1504, 0, 800], [1504, 0, 768]])
@pytest.mark.parametrize("M,N", [(260, 320), (516, 292), (64, 1028)])
@pytest.mark.parametrize("fmt,res", [("e4m3fn", torch.bfloat16), ("e5m2", torch.float32)])
def test_wgrad_tiles(sizes, M, N, fmt, res):
    progress("grouped wgrad %s M=%d N=%d" % (sizes, M, N))
    check_wgrad(sizes, M, N, fmt, res, seed=M + N + sum(sizes))


@pytest.mark.parametrize("sizes", [[800, 0, 1536], [64, 0, 96]])
@pytest.mark.parametrize("N", [320, 292])
def test_wgrad_rare_path(sizes, N):
    def scale(l, ls, r, rs):
        ls[1, ::5], rs[1, :] = 255, 25
        rs[-1, 7:200:3], ls[-1, :] = 255, 25

    def code(l, ls, r, rs):
        l[9, 4 * 130 + 2] = 0x7F
        r[-3, 4 * 270 + 1] = 0xFF

    for patch in (scale, code):
        progress("grouped wgrad, rare path %s N=%d" % (sizes, N))
        check_wgrad(sizes, 260, N, "e4m3fn", torch.bfloat16, 31, patch, per_block=4)
        check_wgrad(sizes, 260, N, "e4m3fn", torch.float32, 32, patch, per_block=4)


@pytest.mark.parametrize("M,N", [(4, 4), (12, 20), (132, 36), (260, 1028)])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_wgrad_empty_groups(M, N, res):
    progress("grouped wgrad, empty groups, M=%d N=%d" % (M, N))
    check_wgrad([0, 32, 0, 0, 64, 0], M, N, "e4m3fn", res, seed=M)
    check_wgrad([0, 1568, 0], M, N, "e4m3fn", res, seed=N)


@pytest.mark.parametrize("patch", [None, scales])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_groups_of_one_and_of_several_128_row_tiles(res, patch):
    """Weights past the caches where a group is one tile; 64 rows on average (32-row
    tiles) and more (128-row ones)."""
    g = np.random.default_rng(12)
    for mean in (64, 68):
        sizes = (4 * g.integers(0, mean // 2, size=40)).tolist()
        sizes[5], sizes[9], sizes[20] = 128, 132, 0
        tail = 40 * mean - sum(sizes) if sum(sizes) < 40 * mean else 4
        progress("grouped rows, 40 groups of %d rows at most, %d rows in all" % (max(sizes), sum(sizes) + tail))
        check_rows(sizes, tail, 96, 2600, "e4m3fn", res, seed=mean, patch=patch, per_block=4)
