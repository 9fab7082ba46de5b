"""GPU tests of the calls around the experts (sort, gather + quantize, combine
and its gradient) against plain references.

The sort and the quantized bytes have to be equal. Sums: the kernels add
`slots` products (the weights' gradient: N) in fp32, each step off by at most
2^-24 of the running magnitude, and round once to the result type (eps / 2 of
it relative; f16 results below 2^-14 by at most 2^-25). References are summed
in 64 bits, so
    |combine - ref|  <= (slots + 1) 2^-24 sum|w y| + eps/2 (|ref| + that) + 2^-25
    |grad_y - ref|   <= (2^-24 + eps/2 (1 + 2^-24)) |ref| + 2^-25
    |grad_w - ref|   <= (N + 8) 2^-24 sum|g y|
"""
import numpy as np
import pytest
import torch

import moe_reference as ref
import mx_microscaling_quantization_amd as mxq
import oracle
import workloads
from conftest import progress

pytestmark = pytest.mark.gpu

IN_T = {"bf16": torch.bfloat16, "f16": torch.float16}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make_ids(T, k, E, seed, missing=0.1, dtype=np.int64):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, size=(T, k))
    ids[g.random((T, k)) < missing] = -1
    return ids.astype(dtype)


def plan_of(ids, E, align=32):
    return mxq.moe_sort(torch.from_numpy(ids).cuda(), E, align)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


# ---- sort --------------------------------------------------------------------

# one workgroup up to 8192 pairs; 8193 and more: two launches; 2^20 pairs and
# more: chunks larger than 4096 pairs
SORTS = [(1, 1, 1, 4), (1, 8, 8, 32), (1, 8, 256, 32), (3, 5, 7, 12), (61, 4, 32, 32), (64, 1, 64, 64), (100, 64, 1000, 4),
         (1024, 8, 128, 32), (1025, 8, 128, 32), (4096, 6, 65, 128), (9000, 3, 1024, 256), (20011, 5, 3, 32),
         (140000, 8, 256, 32)]


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("T,k,E,align", SORTS)
def test_sort(T, k, E, align, dtype):
    progress("sort T=%d k=%d E=%d align=%d %s" % (T, k, E, align, dtype.__name__))
    ids = make_ids(T, k, E, seed=T + k + E, dtype=dtype)
    plan = plan_of(ids, E, align)
    offsets, src, dest = ref.sort(ids, E, align)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.dest.cpu().numpy(), dest)
    assert np.array_equal(plan.src.cpu().numpy(), src)


@pytest.mark.parametrize("T", [100, 5000])
@pytest.mark.parametrize("fill", [0, 3, -1, 4, 1 << 20, -(1 << 31)])
def test_sort_one_expert_or_none(T, fill):
    """Every pair with one expert, or with none (numbers out of range)."""
    ids = np.full((T, 2), fill, np.int32)
    plan = plan_of(ids, 4)
    for got, want in zip(plan, ref.sort(ids, 4, 32)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_wide_ids_are_not_truncated():
    """An int64 number whose low 32 bits name an expert is not that expert."""
    ids = np.array([[1, (1 << 32) + 1], [-(1 << 32), 0]], np.int64)
    for got, want in zip(plan_of(ids, 2, 4), ref.sort(ids, 2, 4)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_no_tokens():
    plan = mxq.moe_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 8)
    assert plan.offsets.tolist() == [0] * 9 and plan.src.numel() == 0 and plan.dest.shape == (0, 2)


# ---- gather and quantize -----------------------------------------------------

def gathered_bits(bits, src, k):
    out = np.zeros((src.size, bits.shape[1]), np.uint16)
    has = (src >= 0) & (src < bits.shape[0] * k)
    out[has] = bits[src[has] // k]
    return out


def check_gather(T, k, E, K, in_dtype, fmt, dim, align=32, dense=True, alt=False, src=None, seed=0):
    bits = workloads.random_bits(T, K, in_dtype, seed=seed + T + K, specials=True)
    plan = plan_of(make_ids(T, k, E, seed), E, align)
    if src is not None:
        plan = mxq.MoEPlan(plan.offsets, torch.from_numpy(src).cuda(), plan.dest)
    x = torch.from_numpy(bits.view(np.int16)).view(IN_T[in_dtype]).cuda()
    rows = plan.src.numel()
    P, F = mxq.axis_view_shape(rows, K, dim)
    data = torch.full((int(np.prod(mxq.data_shape(P, F, fmt))) + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(mxq.scale_image_shape(P, F, dense), dtype=torch.uint8, device="cuda")
    mxq.moe_gather_quantize(x, plan, fmt, dim, data_out=data, scale_out=scale, alt_emax=alt, dense_scale=dense)
    want_d, want_s = oracle.quantize_axis(gathered_bits(bits, plan.src.cpu().numpy(), k), in_dtype, fmt, dim,
                                          alt_emax=alt, layout="dense" if dense else "image")
    got = data.cpu().numpy()
    assert (got[-64:] == 0xA5).all(), "write past the data buffer"
    assert np.array_equal(got[:-64].reshape(want_d.shape), want_d)
    assert np.array_equal(scale.cpu().numpy(), want_s)


GATHERS = [(1, 1, 4, 32), (1, 8, 8, 96), (13, 2, 5, 64), (61, 4, 32, 160), (200, 3, 7, 512), (700, 2, 16, 1056)]


@pytest.mark.parametrize("in_dtype,fmt", [(i, f) for i in ("bf16", "f16") for f in ("e4m3fn", "e5m2", "e2m1")])
@pytest.mark.parametrize("dim", [-1, -2])
@pytest.mark.parametrize("T,k,E,K", GATHERS)
def test_gather_quantize(T, k, E, K, dim, in_dtype, fmt):
    progress("gather_quantize T=%d k=%d E=%d K=%d dim=%d %s->%s" % (T, k, E, K, dim, in_dtype, fmt))
    check_gather(T, k, E, K, in_dtype, fmt, dim)


@pytest.mark.parametrize("K", [1, 2, 3, 6, 30, 127, 130, 261])
def test_gather_quantize_down_any_width(K):
    progress("gather_quantize dim=-2 K=%d" % K)
    check_gather(50, 2, 6, K, "bf16", "e4m3fn", -2)
    check_gather(50, 2, 6, K, "f16", "e2m1", -2)


@pytest.mark.parametrize("dim", [-1, -2])
@pytest.mark.parametrize("dense,alt", [(False, False), (True, True), (False, True)])
def test_gather_quantize_flags(dim, dense, alt):
    check_gather(70, 3, 9, 128, "bf16", "e2m1", dim, dense=dense, alt=alt)
    check_gather(70, 3, 9, 128, "f16", "e4m3fn", dim, dense=dense, alt=alt)


@pytest.mark.parametrize("align", [4, 12, 36])
def test_gather_quantize_along_small_alignment(align):
    check_gather(37, 2, 5, 96, "bf16", "e5m2", -1, align=align)


@pytest.mark.parametrize("dim", [-1, -2])
def test_gather_quantize_entries_out_of_range_are_empty_rows(dim):
    g = np.random.default_rng(3)
    src = g.integers(0, 40, size=96).astype(np.int32)
    src[g.random(96) < 0.4] = np.array([-1, -2, 40, 41, 2 ** 31 - 1, -2 ** 31])[g.integers(0, 6)]
    src[5], src[6], src[77] = 40, 2 ** 31 - 1, -2 ** 31
    check_gather(20, 2, 4, 64, "bf16", "e4m3fn", dim, src=src)


# ---- combine -------------------------------------------------------------------

def tol_out(r, inner, dtype):
    half = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    return inner + half * (np.abs(r) + inner) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def check_combine(T, k, E, N, dtype, weighted=True, seed=0, missing=0.1):
    g = torch.Generator().manual_seed(seed + T + N)
    plan = plan_of(make_ids(T, k, E, seed, missing), E)
    rows = plan.src.numel()
    y = torch.randn((rows, N), generator=g).to(dtype).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    out = mxq.moe_combine(y, plan, w if weighted else None)
    assert out.dtype == dtype and out.shape == (T, N)
    want, mags = ref.combine(host(y), plan.dest.cpu().numpy(), host(w) if weighted else np.ones((T, k)))
    assert (np.abs(host(out) - want) <= tol_out(want, (k + 1) * 2.0 ** -24 * mags, dtype)).all()

    grad = torch.randn((T, N), generator=g).to(dtype).cuda()
    gy, gw = mxq.moe_combine_backward(grad, y, plan, w)
    want_y, want_w, wmags = ref.combine_backward(host(grad), host(y), plan.src.cpu().numpy(),
                                                 plan.dest.cpu().numpy(), host(w))
    assert (np.abs(host(gy) - want_y) <= tol_out(want_y, 2.0 ** -24 * np.abs(want_y), dtype)).all()
    assert (np.abs(host(gw) - want_w) <= (N + 8) * 2.0 ** -24 * wmags).all()


# row lengths about the vector width, odd ones, one and several waves per
# token, several turns; 1 to 13 slots (one and two groups of slots)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,N", [(1, 1, 1, 1), (1, 8, 8, 2), (5, 2, 4, 7), (33, 4, 8, 8), (17, 8, 32, 9),
                                     (40, 3, 6, 64), (12, 13, 16, 130), (9, 9, 5, 515), (6, 2, 3, 2049),
                                     (5, 4, 8, 5000), (3, 11, 7, 8200)])
def test_combine_and_gradient(T, k, E, N, dtype):
    progress("combine T=%d k=%d E=%d N=%d %s" % (T, k, E, N, dtype))
    check_combine(T, k, E, N, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_combine_without_weights(dtype):
    check_combine(29, 4, 6, 100, dtype, weighted=False)


def test_combine_tokens_without_experts():
    check_combine(30, 2, 4, 40, torch.bfloat16, missing=1.0)
    check_combine(30, 2, 4, 40, torch.float32, missing=0.7)


def test_combine_ignores_what_no_pair_reads():
    """Infinities and NaN in rows without a pair, and weights of pairs without
    a row, reach no result."""
    T, k, E, N = 21, 2, 4, 48
    plan = plan_of(make_ids(T, k, E, 5, 0.4), E)
    src, dest = plan.src.cpu(), plan.dest.cpu()
    y = torch.randn((src.numel(), N))
    w = torch.rand((T, k))
    clean = mxq.moe_combine(y.cuda(), plan, w.cuda())
    grad = torch.randn((T, N)).cuda()
    gy0, gw0 = mxq.moe_combine_backward(grad, y.cuda(), plan, w.cuda())
    y[src < 0] = float("nan")
    y[int(np.nonzero(src.numpy() < 0)[0][0])] = float("inf")
    w[dest < 0] = float("nan")
    assert torch.equal(mxq.moe_combine(y.cuda(), plan, w.cuda()), clean)
    gy1, gw1 = mxq.moe_combine_backward(grad, y.cuda(), plan, w.cuda())
    assert torch.equal(gy0, gy1) and torch.equal(gw0, gw1)


def test_combine_entries_out_of_range():
    """dest entries that name no row add nothing and get a zero gradient; src
    entries that name no pair get zero rows."""
    T, k, N, rows = 10, 2, 24, 32
    plan = plan_of(make_ids(T, k, 1, 0, 0.0), 1)
    dest, src = plan.dest.clone(), plan.src.clone()
    assert src.numel() == rows
    bad = torch.tensor([rows, 2 ** 31 - 1, -2, -2 ** 31], dtype=torch.int32)
    for n, b in enumerate(bad):
        row = int(dest[n, 1])
        dest[n, 1] = b
        src[row] = b if b < 0 else T * k + n
    plan = mxq.MoEPlan(plan.offsets, src, dest)
    y, w, grad = torch.randn((rows, N)).cuda(), torch.rand((T, k)).cuda(), torch.randn((T, N)).cuda()
    want, mags = ref.combine(host(y), dest.cpu().numpy(), host(w))
    assert (np.abs(host(mxq.moe_combine(y, plan, w)) - want) <= 3 * 2.0 ** -24 * mags).all()
    gy, gw = mxq.moe_combine_backward(grad, y, plan, w)
    wy, ww, wm = ref.combine_backward(host(grad), host(y), src.cpu().numpy(), dest.cpu().numpy(), host(w))
    assert (np.abs(host(gy) - wy) <= 2.0 ** -24 * np.abs(wy)).all()
    assert (np.abs(host(gw) - ww) <= (N + 8) * 2.0 ** -24 * wm).all()


def test_gradient_against_differences():
    """combine is linear in the weights and in y: a central difference of
    sum(grad * combine) with step 1/2 is exact but for the sums' rounding, at
    most 2 (k + 2) 2^-24 sum|grad| sum|w y|."""
    T, k, E, N = 7, 3, 4, 33
    plan = plan_of(make_ids(T, k, E, 2), E)
    g = torch.Generator().manual_seed(8)
    y = torch.randn((plan.src.numel(), N), generator=g).cuda()
    w, grad = torch.rand((T, k), generator=g).cuda(), torch.randn((T, N), generator=g).cuda()
    gy, gw = mxq.moe_combine_backward(grad, y, plan, w)

    def loss(y, w):
        return (mxq.moe_combine(y, plan, w).double() * grad.double()).sum().item()

    noise = 2 * (k + 2) * 2.0 ** -24 * grad.abs().sum().item() * (w.max() + 0.5).item() * (y.abs().max().item() + 0.5) * k
    for t, j in [(0, 0), (3, 1), (6, 2)]:
        p, m = w.clone(), w.clone()
        p[t, j] += 0.5
        m[t, j] -= 0.5
        assert abs(loss(y, p) - loss(y, m) - gw[t, j].item()) <= noise
    for r, n in [(0, 0), (int(plan.dest.max()), 32), (1, 17)]:
        p, m = y.clone(), y.clone()
        p[r, n] += 0.5
        m[r, n] -= 0.5
        assert abs(loss(p, w) - loss(m, w) - gy[r, n].item()) <= noise


def test_rows_past_32_bits():
    """Row offsets beyond 2^32 elements: y has 2^20 + 64 rows of 4100."""
    N, rows = 4100, (1 << 20) + 64
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    far = [0, 1, rows // 2, rows - 2, rows - 1]
    vals = torch.randn((len(far), N)).to(torch.bfloat16).cuda()
    for n, r in enumerate(far):
        y[r] = vals[n]
    dest = torch.tensor([far], dtype=torch.int32, device="cuda")
    src = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    for n, r in enumerate(far):
        src[r] = n
    plan = mxq.MoEPlan(torch.tensor([0, rows], dtype=torch.int32, device="cuda"), src, dest)
    w = torch.rand((1, len(far))).cuda()
    want, mags = ref.combine(host(vals), np.arange(len(far))[None], host(w))
    got = mxq.moe_combine(y, plan, w)
    assert (np.abs(host(got) - want) <= tol_out(want, 6 * 2.0 ** -24 * mags, torch.bfloat16)).all()
    gy, gw = mxq.moe_combine_backward(got, y, plan, w)
    wy, ww, wm = ref.combine_backward(host(got), host(vals), np.arange(len(far)), np.arange(len(far))[None], host(w))
    for n, r in enumerate(far):
        assert (np.abs(host(gy[r]) - wy[n]) <= tol_out(wy[n], 2.0 ** -24 * np.abs(wy[n]), torch.bfloat16)).all()
    assert (np.abs(host(gw) - ww) <= (N + 8) * 2.0 ** -24 * wm).all()
    assert int(torch.count_nonzero(gy[2:rows // 2])) == 0 and int(torch.count_nonzero(gy[rows // 2 + 1:rows - 2])) == 0


# ---- streams and graphs ----------------------------------------------------------

def test_other_stream_and_repeats():
    """On a stream of its own, behind work that makes its input; equal bits
    every time."""
    ids = torch.from_numpy(make_ids(3000, 4, 32, 1)).cuda()
    base = mxq.moe_sort(ids, 32)
    y0 = torch.randn((base.src.numel(), 256), device="cuda")
    w = torch.rand((3000, 4), device="cuda")
    grad = torch.randn((3000, 256), device="cuda")
    want = mxq.moe_combine(y0 * 2, base, w)
    wy, ww = mxq.moe_combine_backward(grad, y0 * 2, base, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y = y0 * 2
        plan = mxq.moe_sort(ids, 32, stream=s)
        out = mxq.moe_combine(y, plan, w, stream=s)
        gy, gw = mxq.moe_combine_backward(grad, y, plan, w, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        for a, b in ((plan.src, base.src), (plan.dest, base.dest), (out, want), (gy, wy), (gw, ww)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


@pytest.mark.parametrize("T", [512, 4096])
def test_graph_capture(T):
    """Sort (one and two launches), gather and combine captured; the replays see
    new expert numbers and equal the eager results."""
    k, E, K = 4, 16, 256
    ids = torch.from_numpy(make_ids(T, k, E, 1)).cuda()
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    w = torch.rand((T, k), device="cuda")

    def step():
        plan = mxq.moe_sort(ids, E)
        data, scale = mxq.moe_gather_quantize(x, plan)
        y = data.view(torch.float8_e4m3fn).float()[:, :plan.src.numel()]
        y = y.t().contiguous().to(torch.bfloat16)
        out = mxq.moe_combine(y, plan, w)
        return (*plan, data, scale, out, *mxq.moe_combine_backward(out, y, plan, w))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for rep in range(4):
        ids.copy_(torch.from_numpy(make_ids(T, k, E, 10 + rep)))
        for o in outs:
            o.fill_(1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(outs, step())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), "replay %d output %d" % (rep, n)
        _ = (x.float() * 2).sum().item()


# ---- each form, by the rule that picks it -------------------------------------

@pytest.mark.parametrize("in_dtype,fmt", [("bf16", "e4m3fn"), ("f16", "e2m1"), ("f16", "e5m2")])
@pytest.mark.parametrize("T,k,K", [(4100, 2, 4100), (5001, 3, 3460), (300, 2, 520), (8200, 2, 2100)])
def test_gather_quantize_down_orders(T, k, K, in_dtype, fmt):
    """Tiles numbered run by run (x over 32 MiB, up to 8192 tokens, more than one
    slot) and band by band, against quantize_axis on the gathered rows."""
    progress("gather_quantize dim=-2 T=%d k=%d K=%d %s->%s" % (T, k, K, in_dtype, fmt))
    plan = plan_of(make_ids(T, k, 24, T), 24)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = (torch.randn((T, K), generator=g, device="cuda") * 3).to(IN_T[in_dtype])
    rows = torch.where(plan.src[:, None] >= 0, x[plan.src.clamp(min=0).long() // k], torch.zeros((), dtype=x.dtype,
                                                                                                  device="cuda"))
    got = mxq.moe_gather_quantize(x, plan, fmt, dim=-2)
    want = mxq.quantize_axis(rows, fmt, -2, dense_scale=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,k,K", [(3000, 4, 2080), (9001, 2, 96)])
def test_gather_quantize_along_many_tiles(T, k, K):
    plan = plan_of(make_ids(T, k, 24, T), 24)
    x = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    rows = torch.where(plan.src[:, None] >= 0, x[plan.src.clamp(min=0).long() // k], torch.zeros((), dtype=x.dtype,
                                                                                                  device="cuda"))
    for fmt in ("e4m3fn", "e2m1"):
        got = mxq.moe_gather_quantize(x, plan, fmt)
        want = mxq.quantize_axis(rows, fmt, -1, dense_scale=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
