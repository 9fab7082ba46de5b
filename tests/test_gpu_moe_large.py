"""GPU tests of the mixture-of-experts operators on tensors past 2^32 bytes: results and
operands whose last parts lie there, checked in rows at both ends and about each
2^31 bytes. Bounds as in test_gpu_grouped."""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_grouped import compare, dev, host, quantized, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.empty_cache()


def picks(rows, row_bytes, count=4):
    """`count` rows from each multiple of 2^31 bytes on, the first and the last ones."""
    first = {s // row_bytes for s in range(0, rows * row_bytes, 1 << 31)} | {rows - count}
    return np.array(sorted({f + q for f in first for q in range(count) if f + q < rows}))


@pytest.mark.parametrize("K,res", [(32, torch.bfloat16), (1056, torch.bfloat16), (32, torch.float32)])
def test_grouped_rows_past_32_bits(K, res):
    """[rows, 4096] results of 5 GiB: 128- and 256-row tiles; 40 rows cleared past
    the last group, beyond 2^32 bytes too."""
    N, es = 4096, 2 if res == torch.bfloat16 else 4
    rows = (5 << 30) // (N * es)
    progress("grouped rows, %d x %d results, K=%d" % (rows, N, K))
    l0, ls0 = quantized(1024, K, -1, "e4m3fn", 1)
    reps = rows // 1024
    l = dev(l0).view(K // 4, 4096).repeat(1, reps)       # row r is row r % 1024 of l0
    ls = dev(ls0).repeat(1, reps)
    rows = reps * 1024
    r, rs = (np.stack(t) for t in zip(*[quantized(K, N, -2, "e4m3fn", g) for g in range(3)]))
    off = np.array([0, 1000, rows // 2, rows - 40], np.int32)
    out = torch.full((rows, N), 7.0, dtype=res, device="cuda")
    mxq.grouped_scaled_matmul(l, ls, dev(r), dev(rs), dev(off), "e4m3fn", res, out=out)
    L = values(l0, ls0, "e4m3fn")
    assert int(torch.count_nonzero(out[rows - 40:])) == 0
    at = picks(rows - 40, N * es)
    for g in range(3):
        here = at[(at >= off[g]) & (at < off[g + 1])]
        if len(here):
            compare(host(out[torch.from_numpy(here).cuda()]), L[:, here % 1024], values(r[g], rs[g], "e4m3fn"), res)
    # and every other row is one of these three groups' rows of that operand
    for a, b in ((1024, rows // 2), ((rows // 2 + 1023) // 1024 * 1024, rows - 1024)):
        span = out[a:b - (b - a) % 1024].view(-1, 1024, N)
        assert torch.equal(span, span[:1].expand_as(span))


def test_grouped_weights_past_32_bits():
    """70 experts of 8192 x 8192: the last ones' weights lie past 2^32 bytes."""
    E, K, N = 70, 8192, 8192
    progress("grouped rows, %d experts of %d x %d" % (E, K, N))
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    r = torch.randint(0, 256, (E, K // 4, 4 * N), dtype=torch.uint8, device="cuda", generator=g)
    r.bitwise_and_(0xBF)        # finite: the top bit of the exponent is off
    rs = torch.randint(118, 134, (E, K // 32, N), dtype=torch.uint8, device="cuda", generator=g)
    l, ls = quantized(E * 8, K, -1, "e4m3fn", 9)
    off = np.arange(E + 1, dtype=np.int32) * 8
    out = mxq.grouped_scaled_matmul(dev(l), dev(ls), r, rs, dev(off), "e4m3fn", torch.float32)
    L = values(l, ls, "e4m3fn")
    cols = np.array([0, 1, 4095, 8190, 8191])
    for e in (0, 31, 32, 63, 64, E - 1):
        w = r[e].view(K // 4, N, 4)[:, torch.from_numpy(cols).cuda()].reshape(K // 4, -1).cpu().numpy()
        ws = rs[e][:, torch.from_numpy(cols).cuda()].cpu().numpy()
        compare(host(out[8 * e:8 * e + 8])[:, cols], L[:, 8 * e:8 * e + 8], values(w, ws, "e4m3fn"), torch.float32)


@pytest.mark.parametrize("size", [64, 768])
def test_grouped_wgrad_past_32_bits(size):
    """40 gradients of 8192 x 8192 bf16 (5 GiB), some of them of empty groups; 128-
    and 256-row tiles."""
    E, M, N = 40, 8192, 8192
    progress("grouped wgrad, %d groups of %d rows, %d x %d" % (E, size, M, N))
    sizes = np.full(E, size)
    sizes[[1, 33, 39]], sizes[[2, 34, 38]] = 0, 2 * size
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = int(off[-1])
    l0, ls0 = quantized(rows, 1024, -2, "e4m3fn", 5)     # column m is column m % 1024
    r0, rs0 = quantized(rows, 1024, -2, "e4m3fn", 6)
    out = torch.full((E, M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    mxq.grouped_scaled_matmul_wgrad(dev(l0).repeat(1, 8), dev(ls0).repeat(1, 8), dev(r0).repeat(1, 8),
                                    dev(rs0).repeat(1, 8), dev(off), "e4m3fn", torch.bfloat16, out=out)
    L, R = values(l0, ls0, "e4m3fn"), values(r0, rs0, "e4m3fn")
    for g in range(E):
        part = out[g].view(8, 1024, 8, 1024)
        first = part[0, :, 0]
        assert torch.equal(part, first[None, :, None].expand_as(part))
        if sizes[g] == 0:
            assert int(torch.count_nonzero(first)) == 0
        elif g in (0, 15, 16, 32, 34, 38):
            m = np.array([0, 5, 600, 1023])
            a, b = off[g], off[g + 1]
            compare(host(first[torch.from_numpy(m).cuda()]), L[a:b, m], R[a:b], torch.bfloat16)


@pytest.mark.parametrize("dim", [-1, -2])
def test_gather_quantize_past_32_bits(dim):
    """[540000, 8192] bf16 input and codes past 2^32 bytes, against quantize_axis on
    the gathered rows of some runs of 32."""
    T, K = 540000, 8192
    progress("gather_quantize T=%d K=%d dim=%d" % (T, K, dim))
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    for a in range(0, T, 54000):
        x[a:a + 54000] = torch.randn((54000, K), device="cuda")
    rows = T
    src = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    src[rows - 20:rows - 10] = -1
    plan = mxq.MoEPlan(torch.tensor([0, rows], dtype=torch.int32, device="cuda"), src,
                       torch.full((T, 1), -1, dtype=torch.int32, device="cuda"))
    data, scale = mxq.moe_gather_quantize(x, plan, "e4m3fn", dim)
    starts = sorted({a // 32 * 32 for s in range(0, rows * K, 1 << 30) for a in (s // K, s // K + 32)} |
                    {rows - 32, rows // 64 * 32})
    for a in starts:
        here = src[a:a + 32].long()
        part = torch.where(here[:, None] >= 0, x[here.clamp(min=0)], torch.zeros((), dtype=x.dtype, device="cuda"))
        want_d, want_s = mxq.quantize_axis(part, "e4m3fn", dim, dense_scale=True)
        if dim == -1:
            got_d, got_s = data[:, 4 * a:4 * a + 128], scale[:, a:a + 32]
        else:
            got_d, got_s = data[a // 4:a // 4 + 8], scale[a // 32:a // 32 + 1]
        assert torch.equal(got_d.contiguous(), want_d) and torch.equal(got_s.contiguous(), want_s), a
