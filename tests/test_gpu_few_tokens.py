"""GPU tests of the mixture-of-experts layer for a few tokens against the layer in 64
bits on the same quantized weights.

Bounds, for unit u = 2^-24 and a result y = sum_j w_j sum_f h_f W2_f with h = act(z):
a product's fp32 sum of K terms is off by at most (K + 10) u of the sum of its terms'
magnitudes (each addition by half a step of a partial sum; 8 waves' sums are added on top).
The exponential's argument z log2(e) is off by two roundings, 2 |z| u in the
exponential's relative error, and the steps from there to silu by 7 u more (exponential
and reciprocal a whole step each, sum, product): (2 |z| + 8) u of its magnitude; its slope is at most 1.1 in magnitude, so an error d in z
gives at most 1.1 d. h is kept to 2^-17 of its value (two bf16 numbers: half a step of 2^-8
of what the first one leaves, at most 2^-9 of the value). The result is rounded once,
by at most half a step of its type.
"""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
import oracle
import workloads
from conftest import progress
from test_gpu_fp4 import values
from test_gpu_grouped import dev, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def weights_of(E, K, C, fmt, seed):
    """[E, ..] codes and dense scales of normal [K, C] weights."""
    g = np.random.default_rng(seed)
    out = []
    for _ in range(E):
        w = (g.normal(size=(K, C)) / np.sqrt(max(K, 1))).astype(np.float32)
        bits = workloads.f32_to_bf16_bits(w)
        out.append(oracle.quantize_axis(bits, "bf16", fmt, -2, layout="dense"))
    return tuple(np.stack(t) for t in zip(*out))


def reference(x, ids, weights, w1, w2, act):
    """(out, bound before rounding) in float64; w1 and w2 as value matrices per expert."""
    T, k = ids.shape
    N = w2[0].shape[1]
    out, bound = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < len(w1):
                continue
            z, zm = x[t] @ w1[e], np.abs(x[t]) @ np.abs(w1[e])
            dz = (x.shape[1] + 10) * U * zm
            F = w2[e].shape[0]
            gate, dg = z[:F], dz[:F]
            s = gate / (1.0 + np.exp(-gate))
            ds = 1.1 * dg + (2 * np.abs(gate) + 8) * U * np.abs(s)
            if act == "swiglu":
                h = s * z[F:]
                dh = ds * np.abs(z[F:]) + np.abs(s) * dz[F:] + ds * dz[F:] + U * np.abs(h)
            else:
                h, dh = s, ds
            dh = dh + 2.0 ** -17 * (np.abs(h) + dh)
            y, ym = h @ w2[e], (np.abs(h) + dh) @ np.abs(w2[e])
            wt = float(weights[t, j])
            out[t] += wt * y
            bound[t] += abs(wt) * (dh @ np.abs(w2[e]) + (F + 10) * U * ym) + (k + 2) * U * abs(wt) * ym
    return out, bound


def case(T, k, E, K, F, N, fmt="e2m1", act="swiglu", dtype=torch.bfloat16, id_dtype=torch.int64, ids=None, patch=None,
         seed=0, missing=0.0):
    progress("few tokens T=%d k=%d E=%d K=%d F=%d N=%d %s %s %s" % (T, k, E, K, F, N, fmt, act, dtype))
    g = np.random.default_rng(seed + T + 7 * E + K)
    if ids is None:
        ids = np.stack([g.permutation(max(E, k))[:k] for _ in range(T)]) if T else np.zeros((0, k), np.int64)
        ids = np.where(g.random(ids.shape) < missing, -1, ids)
    x = torch.from_numpy(g.normal(size=(T, K))).to(dtype)
    wt = torch.from_numpy(g.random((T, k)).astype(np.float32))
    w1 = weights_of(E, K, F * (2 if act == "swiglu" else 1), fmt, seed + 1)
    w2 = weights_of(E, F, N, fmt, seed + 2)
    if patch:
        patch(x, w1, w2)
    call = (x.cuda(), torch.from_numpy(ids).to(id_dtype).cuda(), wt.cuda(), dev(w1[0]), dev(w1[1]), dev(w2[0]),
            dev(w2[1]), fmt, act)
    return call, (host(x), ids, wt.numpy().astype(np.float64), [values(a, b, fmt) for a, b in zip(*w1)],
                  [values(a, b, fmt) for a, b in zip(*w2)], act)


def check(call, plain):
    x, N = call[0], call[6].shape[2]
    room = torch.full((x.shape[0] * N + 64,), 7.0, dtype=x.dtype, device="cuda")
    mxq.moe_few_tokens(*call, out=room[:x.shape[0] * N].view(-1, N))
    got = host(room)
    assert (got[x.shape[0] * N:] == 7).all()
    got = got[:x.shape[0] * N].reshape(-1, N)
    with np.errstate(all="ignore"):
        want, bound = reference(*plain)
    step = STEP[x.dtype]
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fin)
    off = np.abs(got - want) - (bound + step * (np.abs(want) + bound) + tiny)
    assert (off[fin] <= 0).all(), "worst %g over the bound" % off[fin].max()
    return got


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3fn", "e5m2"])
@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,E,K,F,N", [(1, 1, 1, 32, 32, 4), (1, 2, 4, 64, 32, 36), (3, 2, 8, 288, 160, 132),
                                         (16, 4, 8, 96, 96, 64), (61, 6, 9, 64, 96, 100), (40, 2, 2, 544, 288, 260)])
def test_layer(T, k, E, K, F, N, fmt, act, dtype):
    check(*case(T, k, E, K, F, N, fmt, act, dtype))


@pytest.mark.parametrize("T,k,E", [(1, 8, 128), (13, 3, 1024), (128, 8, 5), (1024, 1, 3), (16, 64, 70), (70, 1, 1),
                                   (33, 1, 1), (17, 1, 1), (200, 1, 2)])
@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
def test_routes(T, k, E, id_dtype):
    """From one pair to the most there may be, one expert with all of them, experts past
    the first mask word, ids outside the experts."""
    if k > E:
        ids = np.random.default_rng(T).integers(-1, E + 1, size=(T, k))
        check(*case(T, k, E, 32, 32, 12, id_dtype=id_dtype, ids=ids))
    else:
        check(*case(T, k, E, 32, 32, 12, id_dtype=id_dtype))
        check(*case(T, k, E, 64, 32, 8, id_dtype=id_dtype, missing=0.4, seed=3))


def test_experts_named_twice_and_tokens_without_any():
    ids = np.array([[2, 2, 2], [-1, -1, -1], [0, 5, 0], [7, -3, 1], [2 ** 31 - 1, 1, -2 ** 31]])
    got = check(*case(5, 3, 4, 64, 64, 20, ids=ids))
    assert (got[1] == 0).all()
    far = ids.copy()
    far[3] = [2 ** 40, 2 ** 32 + 1, -2 ** 62]
    got = check(*case(5, 3, 4, 64, 64, 20, ids=far))
    assert (got[3] == 0).all()
    got = check(*case(5, 3, 4, 64, 64, 20, ids=np.full((5, 3), -1)))
    assert (got == 0).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3fn", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scale_255(fmt, dtype):
    """255 stands for 2^128, in either product."""
    def zeros(x, w1, w2):
        x[:, 32:64] = 0.0
        w1[1][:, 1, ::5] = 255
        w2[1][:, 0, ::3] = 255
        x[2:] = 0.0

    with np.errstate(all="ignore"):
        call, plain = case(6, 2, 2, 96, 32, 36, fmt, "swiglu", dtype, patch=zeros)
    got = host(mxq.moe_few_tokens(*call))
    assert (got[2:] == 0).all()

    def small(x, w1, w2):      # small activations into a down projection with weights of 2^128
        x[:] = x * 2.0 ** -12
        w1[1][:] = np.where(w1[1] > 60, w1[1] - 60, 1)
        w2[1][:, 0, ::3] = 255

    # weights of 2^128 whose columns' activations meet small weights. The first product has to
    # stay in fp32's range: an e5m2 block's largest value is 57344 * 2^128, below 2^144,
    # so x up to 4 times 2^-30 gives at most 32 * 2^116.
    def up(x, w1, w2):
        x[:, 32:64] = x[:, 32:64] * 2.0 ** -30
        w1[1][:, 1, 3] = 255
        w2[1][:] = np.where(w2[1] > 100, w2[1] - 100, 1)

    if dtype == torch.bfloat16:     # (f16 has no such results)
        check(*case(6, 2, 2, 96, 32, 36, fmt, "silu", dtype, patch=small))
        check(*case(6, 2, 2, 96, 32, 36, fmt, "silu", dtype, patch=up))


def test_infinities_and_nan_stay_with_their_token():
    call, _ = case(9, 2, 4, 96, 64, 68)
    want = mxq.moe_few_tokens(*call)
    for bad in (float("inf"), float("nan"), -float("inf")):
        x = call[0].clone()
        x[4, 17] = bad
        got = mxq.moe_few_tokens(x, *call[1:])
        assert not bool(torch.isfinite(got[4]).all())
        keep = [t for t in range(9) if t != 4]
        assert torch.equal(got[keep], want[keep])


def test_no_tokens_and_no_contraction():
    call, _ = case(0, 2, 4, 64, 32, 8)
    assert mxq.moe_few_tokens(*call).shape == (0, 8)
    call, _ = case(3, 2, 4, 0, 32, 8)
    assert int(torch.count_nonzero(mxq.moe_few_tokens(*call))) == 0
    call, _ = case(3, 2, 4, 64, 0, 8)
    assert int(torch.count_nonzero(mxq.moe_few_tokens(*call))) == 0


def test_against_the_sorted_calls():
    """The same layer through sort, gather, grouped products and combine on FP8 activations:
    within what two roundings of the activations to e4m3 (2^-4 each, in the norm far
    less) leave."""
    T, k, E, K, F, N = 50, 2, 6, 256, 128, 192
    call, plain = case(T, k, E, K, F, N, "e2m1", "silu", seed=5)
    x, ids, wt, w1, s1, w2, s2 = call[:7]
    plan = mxq.moe_sort(ids, E)
    z = mxq.grouped_scaled_matmul_fp4(*mxq.moe_gather_quantize(x, plan), w1, s1, plan.offsets)
    a = torch.nn.functional.silu(z)
    y = mxq.grouped_scaled_matmul_fp4(*mxq.quantize_axis(a, "e4m3fn", -1, dense_scale=True), w2, s2, plan.offsets)
    want = host(mxq.moe_combine(y, plan, wt))
    got = check(call, plain)
    assert np.linalg.norm(got - want) <= (2.0 ** -4 + 2.0 ** -4) * np.linalg.norm(got)


def test_other_stream_graph_and_repeats():
    a, _ = case(16, 4, 8, 288, 160, 132)
    b, _ = case(40, 2, 5, 96, 96, 64, "e4m3fn", "silu", torch.float16, torch.int32)

    def run(**kw):
        return mxq.moe_few_tokens(*a, **kw), mxq.moe_few_tokens(*b, **kw)

    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):     # two calls at once, on two streams
        got, here = run(stream=s), run()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(p, q) for p, q in zip(got + here, want + want))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        graphs.append((g, got))
    for _ in range(4):
        for g, got in graphs:
            for t in got:
                t.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(run(), want))
    # other routes and activations in the captured call's tensors
    g, got = graphs[0]
    x, ids = a[0], a[1]
    x.copy_(torch.randn_like(x))
    ids.copy_((ids + 1) % 8)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], mxq.moe_few_tokens(*a))


def test_results_given_by_the_caller_count_a_version():
    call, _ = case(3, 2, 4, 64, 32, 8)
    out = torch.empty((3, 8), dtype=torch.bfloat16, device="cuda")
    v = out._version
    assert mxq.moe_few_tokens(*call, out=out) is out and out._version == v + 1
