"""GPU tests of the layer for a few tokens at sizes of real layers: more than 256 workgroups in
either kernel (four waves share a contraction then, eight below), contractions of several rounds
of every wave's blocks and a rest, one to four tiles of pairs an expert. Sampled tokens and
columns against the layer in 64 bits; bounds as in test_gpu_few_tokens.
"""
import ctypes

import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_few_tokens import STEP, U, weights_of
from test_gpu_fp4 import values
from test_gpu_grouped import dev, host

pytestmark = pytest.mark.gpu


def skewed(T, k, E, first, seed):
    """Experts of T tokens; the first of them has `first` of the tokens, the others even shares."""
    g = np.random.default_rng(seed)
    ids = np.stack([1 + g.permutation(E - 1)[:k] for _ in range(T)])
    ids[g.permutation(T)[:first], 0] = 0
    return ids


def experts_of(E, K, C, fmt, seed):
    """As weights_of; expert e is one of three matrices with its columns moved on by e."""
    base, scale = weights_of(3, K, C, fmt, seed)
    codes = base.reshape(3, K // 4, C, -1)
    return (np.stack([np.roll(codes[e % 3], e, 1).reshape(K // 4, -1) for e in range(E)]),
            np.stack([np.roll(scale[e % 3], e, 1) for e in range(E)]))


def sampled(x, ids, weights, w1, w2, fmt, act, tokens, cols):
    """(out, bound before rounding) of these tokens and columns in float64."""
    F, gated = w2[1].shape[1] * 32, act == "swiglu"
    out, bound = np.zeros((len(tokens), len(cols))), np.zeros((len(tokens), len(cols)))
    per = 2 if fmt == "e2m1" else 4
    for e in np.unique(ids[tokens]):
        t, j = np.nonzero(ids[tokens] == e)
        first = values(w1[0][e], w1[1][e], fmt)
        rows = x[tokens][t]
        K = rows.shape[1]
        z, dz = rows @ first, (K + 10) * U * (np.abs(rows) @ np.abs(first))
        gate, dg = z[:, :F], dz[:, :F]
        s = gate / (1.0 + np.exp(-gate))
        ds = 1.1 * dg + (2 * np.abs(gate) + 8) * U * np.abs(s)
        if gated:
            h = s * z[:, F:]
            dh = ds * np.abs(z[:, F:]) + np.abs(s) * dz[:, F:] + ds * dz[:, F:] + U * np.abs(h)
        else:
            h, dh = s, ds
        dh = dh + 2.0 ** -17 * (np.abs(h) + dh)
        codes = w2[0][e].reshape(F // 4, -1, per)[:, cols].reshape(F // 4, -1)
        second = values(codes, w2[1][e][:, cols], fmt)
        y, ym = h @ second, (np.abs(h) + dh) @ np.abs(second)
        wt = weights[tokens][t, j].astype(np.float64)[:, None]
        np.add.at(out, t, wt * y)
        np.add.at(bound, t, np.abs(wt) * (dh @ np.abs(second) + (F + 10) * U * ym) + (ids.shape[1] + 2) * U * np.abs(wt) * ym)
    return out, bound


def check(T, k, E, K, F, N, fmt, act, dtype, first, seed):
    progress("few tokens T=%d k=%d E=%d K=%d F=%d N=%d %s %s %s" % (T, k, E, K, F, N, fmt, act, dtype))
    g = np.random.default_rng(seed)
    ids = skewed(T, k, E, first, seed)
    x = torch.from_numpy(g.normal(size=(T, K))).to(dtype)
    wt = g.random((T, k)).astype(np.float32)
    w1 = experts_of(E, K, F * (2 if act == "swiglu" else 1), fmt, seed + 1)
    w2 = experts_of(E, F, N, fmt, seed + 2)
    call = (x.cuda(), dev(ids), dev(wt), dev(w1[0]), dev(w1[1]), dev(w2[0]), dev(w2[1]), fmt, act)
    out = mxq.moe_few_tokens(*call)
    for _ in range(3):          # the exchange between workgroups does not show in the result
        assert torch.equal(out, mxq.moe_few_tokens(*call))
    tokens = np.unique(np.concatenate([[0, T - 1], np.nonzero((ids == 0).any(1))[0][:3], g.permutation(T)[:4]]))
    cols = np.unique(np.concatenate([[0, 1, 62, 63, 64, N - 65, N - 2, N - 1], g.integers(0, N, 24)]))
    want, bound = sampled(host(x), ids, wt, w1, w2, fmt, act, tokens, cols)
    got = host(out)[np.ix_(tokens, cols)]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    off = np.abs(got - want) - (bound + STEP[dtype] * (np.abs(want) + bound) + tiny)
    assert (off <= 0).all(), "worst %g over the bound" % off.max()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3fn", "e5m2"])
@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_more_workgroups_than_cus(act, fmt):
    """33 experts x 9 and 10 column tiles; 65 and 18 blocks for four waves."""
    check(16, 4, 33, 2080, 576, 580, fmt, act, torch.bfloat16, 5, 1)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3fn", "e5m2"])
def test_two_tiles_of_pairs(fmt):
    """17 experts x 17 column tiles, some 24 pairs each; f16 rows."""
    check(67, 6, 17, 2336, 1088, 1060, fmt, "silu", torch.float16, 25, 2)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3fn", "e5m2"])
@pytest.mark.parametrize("act,dtype", [("swiglu", torch.bfloat16), ("silu", torch.float16)])
def test_four_tiles_of_pairs(act, dtype, fmt):
    """An expert with all 100 tokens (64 pairs, 32 and a rest) among others of 34 to 53 pairs."""
    check(100, 8, 17, 1312, 1088, 1060, fmt, act, dtype, 100, 3)


@pytest.mark.parametrize("T,k,F,N", [(1024, 1, 32, 4), (333, 3, 32, 68), (16, 64, 64, 132), (1, 1, 32, 4)])
def test_workspace_is_all_that_is_written(T, k, F, N):
    """A workspace of the queried size, filled with other bytes before: what lies behind it
    stays, and the result is the same as with one of the binding's."""
    progress("few tokens, a workspace of the caller's: T=%d k=%d F=%d N=%d" % (T, k, F, N))
    lib, E, K = mxq.load(), 5, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    wt = torch.rand((T, k), generator=g, device="cuda")
    w1, w2 = (tuple(map(dev, weights_of(E, a, b, "e4m3fn", 3))) for a, b in ((K, F), (F, N)))
    want = mxq.moe_few_tokens(x, ids, wt, *w1, *w2, "e4m3fn", "silu")
    size = lib.mxq_moe_few_tokens_workspace_bytes(T, k, F, N)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full_like(want, 3.0)
    rc = lib.mxq_moe_few_tokens(x.data_ptr(), T, K, 0, ids.data_ptr(), 4, wt.data_ptr(), k, E, w1[0].data_ptr(),
                                w1[1].data_ptr(), w2[0].data_ptr(), w2[1].data_ptr(), F, N,
                                mxq.OUT_DTYPES["e4m3fn"], mxq.ACTIVATIONS["silu"], room.data_ptr(), out.data_ptr(),
                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert bool((room[size:] == 0xA5).all())
