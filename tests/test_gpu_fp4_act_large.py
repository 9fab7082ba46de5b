"""GPU tests of the products with 4-bit weights, the layer for a few tokens and the
activations between products on tensors past 2^32 bytes: against exact sums in some
rows and columns (bounds as in test_gpu_grouped), or, bit by bit, against the same call
on the part that lies there."""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_fp4 import values
from test_gpu_grouped import compare, dev, host, quantized
from test_gpu_moe_large import picks

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.empty_cache()


def random_bytes(*shape, low=0, high=256, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(low, high, shape, dtype=torch.uint8, device="cuda", generator=g)


# 1024 groups of 64 rows: streamed; short and longer contractions: the square tiles
@pytest.mark.parametrize("groups,rows,N,K,fmt", [(1024, 65536, 40960, 32, "e4m3fn"), (3, 655360, 4096, 32, "e2m1"),
                                                 (3, 655360, 4096, 1056, "e5m2")])
def test_grouped_results(groups, rows, N, K, fmt):
    progress("fp4 grouped, %d rows in %d groups, %d x %d, %s" % (rows, groups, K, N, fmt))
    l0, ls0 = quantized(1024, K, -1, fmt, 1)
    l = dev(l0).repeat(1, rows // 1024)         # row r is row r % 1024 of l0
    ls = dev(ls0).repeat(1, rows // 1024)
    r, rs = (np.stack(t) for t in zip(*[quantized(K, N, -2, "e2m1", g) for g in range(min(groups, 3))]))
    which = np.arange(groups) % len(r)
    off = (np.arange(groups + 1) * (rows // groups // 4 * 4)).astype(np.int32)
    off[-1] = rows - 40
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    at = torch.from_numpy(which).cuda()
    mxq.grouped_scaled_matmul_fp4(l, ls, dev(r)[at], dev(rs)[at], dev(off), fmt, torch.bfloat16, out=out)
    assert int(torch.count_nonzero(out[rows - 40:])) == 0
    L = values(l0, ls0, fmt)
    R = [values(r[g], rs[g], "e2m1") for g in range(len(r))]
    rows_at = picks(rows - 40, 2 * N)
    group = np.searchsorted(off, rows_at, "right") - 1
    for g in np.unique(group):
        here = rows_at[group == g]
        compare(host(out[torch.from_numpy(here).cuda()]), L[:, here % 1024], R[which[g]], torch.bfloat16)
    if groups == 3:                             # and every other row is one of these
        for a, b in ((0, off[1] // 1024 * 1024), (-(-off[2] // 1024) * 1024, rows - 1024)):
            span = out[int(a):int(b)].view(-1, 1024, N)
            assert torch.equal(span, span[:1].expand_as(span))


@pytest.mark.parametrize("per,fmt", [(8, "e4m3fn"), (128, "e4m3fn"), (512, "e2m1")])
def test_grouped_weights(per, fmt):
    """140 experts of 8192 x 8192 in e2m1."""
    E, K, N = 140, 8192, 8192
    progress("fp4 grouped, %d experts of %d x %d, %d rows each, %s" % (E, K, N, per, fmt))
    r = random_bytes(E, K // 4, 2 * N, seed=3)
    rs = random_bytes(E, K // 32, N, low=118, high=134, seed=4)
    l0, ls0 = quantized(per, K, -1, fmt, 9)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * per
    out = mxq.grouped_scaled_matmul_fp4(dev(l0).repeat(1, E), dev(ls0).repeat(1, E), r, rs, off, fmt, torch.float32)
    rows = np.unique([0, 5, per // 2, per - 1])
    L = values(l0, ls0, fmt)[:, rows]
    cols = torch.tensor([0, 1, 4095, 8190, 8191], device="cuda")
    for e in (0, 63, 64, 127, 128, E - 1):
        w = r[e].view(K // 4, N, 2)[:, cols].reshape(K // 4, -1).cpu().numpy()
        got = out[e * per + torch.from_numpy(rows).cuda()][:, cols]
        compare(host(got), L, values(w, rs[e][:, cols].cpu().numpy(), "e2m1"), torch.float32)


@pytest.mark.parametrize("fmt,K", [("e4m3fn", 128), ("e2m1", 288)])
def test_dense_rows(fmt, K):
    """Nearly as many rows as a call takes, activations past 2^32 bytes."""
    M, N = 33553408, 32
    progress("fp4 product %d x %d x %d, %s" % (M, K, N, fmt))
    l0, ls0 = quantized(1024, K, -1, fmt, 1)
    r, rs = quantized(K, N, -2, "e2m1", 2)
    out = mxq.scaled_matmul_fp4(dev(l0).repeat(1, M // 1024), dev(ls0).repeat(1, M // 1024), dev(r), dev(rs), fmt,
                                torch.bfloat16, dense_scale=True)
    span = out.view(-1, 1024, N)
    assert torch.equal(span, span[:1].expand_as(span))
    compare(host(span[-1]), values(l0, ls0, fmt), values(r, rs, "e2m1"), torch.bfloat16)


def test_dense_weights():
    """A product of one row with a matrix of 2^32 bytes and more."""
    K, N, M = 65536, 139264, 1
    progress("fp4 product %d x %d x %d" % (M, K, N))
    r = random_bytes(K // 4, 2 * N, seed=5)
    rs = random_bytes(K // 32, N, low=118, high=134, seed=6)
    l, ls = quantized(M, K, -1, "e4m3fn", 9)
    out = mxq.scaled_matmul_fp4(dev(l), dev(ls), r, rs, "e4m3fn", torch.float32, dense_scale=True)
    cols = torch.tensor([0, 1, N // 2, N - 2, N - 1], device="cuda")
    w = r.view(K // 4, N, 2)[:, cols].reshape(K // 4, -1).cpu().numpy()
    compare(host(out[:, cols]), values(l, ls, "e4m3fn"), values(w, rs[:, cols].cpu().numpy(), "e2m1"), torch.float32)


@pytest.mark.parametrize("fmt,E", [("e4m3fn", 70), ("e2m1", 140)])
def test_few_tokens_weights(fmt, E):
    """Both matrices of the last experts past 2^32 bytes; the same as with the used
    experts alone (as many of them are in use, so the sums are in the same order)."""
    K = F = N = 8192
    progress("few tokens, %d experts of %d x %d, %s" % (E, K, F, fmt))
    cb = 2 if fmt == "e2m1" else 4
    mask = 0xFF if fmt == "e2m1" else 0xBF      # finite: the top bit of the exponent is off
    w1 = random_bytes(E, K // 4, cb * F, seed=1).bitwise_and_(mask)
    w2 = random_bytes(E, F // 4, cb * N, seed=2).bitwise_and_(mask)
    s1 = random_bytes(E, K // 32, F, low=116, high=122, seed=3)
    s2 = random_bytes(E, F // 32, N, low=116, high=122, seed=4)
    pick = [0, E // 2, E - 2, E - 1]
    ids = torch.tensor([pick, pick[::-1]], device="cuda")
    small = torch.tensor([[0, 1, 2, 3], [3, 2, 1, 0]], device="cuda")
    x = torch.randn((2, K), device="cuda").to(torch.bfloat16)
    w = torch.rand((2, 4), device="cuda")
    got = mxq.moe_few_tokens(x, ids, w, w1, s1, w2, s2, fmt, "silu")
    want = mxq.moe_few_tokens(x, small, w, *(t[pick].contiguous() for t in (w1, s1, w2, s2)), fmt, "silu")
    assert bool(torch.isfinite(got).all()) and int(torch.count_nonzero(got)) > N
    assert torch.equal(got, want)


@pytest.mark.parametrize("act,R,F", [("silu", 540032, 8192), ("swiglu", 540032, 4096), ("swiglu", 2080, 1081344)])
def test_activations(act, R, F):
    W = 2 * F if act == "swiglu" else F
    progress("activations %s %d x %d" % (act, R, F))
    z = torch.empty((R, W), dtype=torch.bfloat16, device="cuda")
    grad = torch.empty((R, F), dtype=torch.bfloat16, device="cuda")
    for t in (z, grad):
        for a in range(0, R, R // 16):
            t[a:a + R // 16].normal_()
    (data, scale), (saved, saved_scale) = mxq.act_quantize(z, act)
    got = mxq.act_quantize_backward(grad, saved, saved_scale, act)
    for a in sorted({s // (2 * W) // 32 * 32 for s in range(0, 2 * R * W, 1 << 31)} | {R - 32}):
        b = a + 32
        (d, s), (k, ks) = mxq.act_quantize(z[a:b], act)
        assert torch.equal(data.view(F // 4, R, 4)[:, a:b].reshape(d.shape), d), a
        assert torch.equal(scale[:, a:b], s) and torch.equal(saved[a:b], k), a
        assert torch.equal(saved_scale[a // 8:b // 8], ks), a
        want = mxq.act_quantize_backward(grad[a:b], k, ks, act)
        assert torch.equal(got.rows[0].view(W // 4, R, 4)[:, a:b].reshape(want.rows[0].shape), want.rows[0]), a
        assert torch.equal(got.rows[1][:, a:b], want.rows[1]), a
        for x, y in ((got.cols, want.cols), (got.h, want.h)):
            assert torch.equal(x[0][a // 4:b // 4], y[0]) and torch.equal(x[1][a // 32:b // 32], y[1]), a
