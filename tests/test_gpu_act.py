"""GPU tests of the activation between products (quantized result, input kept in 8 bits)
and of its backward pass.

The kept input is the quantize of z itself: equal bytes. The result h and the gradients
are computed in fp32 and rounded to 16 bits before they are quantized, so their bytes are
those of the oracle's quantize wherever fp32's error cannot move a value over a rounding
border (zeros of either sign taken as equal). With u = 2^-24: the exponential's argument is off by two roundings (2 |z| u in
the exponential), exponential and reciprocal by a step of 2 u each, sums and products by
u, so s = 1 / (1 + e^-z) is off by (2 |z| + 5) u of itself, silu by (2 |z| + 8) u, and
its slope s + silu(z) (1 - s) by (2 |z| + 10) u (s + 2 |silu|). Rounding and quantizing keep
an order, so a block whose codes and scale are the same at both ends of the intervals
of that width has to have them; in the others the scale is the oracle's or a neighbour, and a value within half
a step of the format at that scale, and the interval, of what it stands for (values past
the largest code, of which a block's top binade has some, become that code). Those others are few.
"""
import numpy as np
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
import oracle
from conftest import progress
from test_gpu_fp4 import values
from test_gpu_grouped import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NAMES = {torch.bfloat16: "bf16", torch.float16: "f16"}
# half a step relative to the value, exponent of the largest code, the largest code
FORMAT = {"e4m3fn": (2.0 ** -4, 8, 448.0), "e5m2": (2.0 ** -3, 15, 57344.0), "e2m1": (2.0 ** -2, 2, 6.0)}


def bits(t):
    return t.contiguous().view(torch.int16).numpy().view(np.uint16)


def rounded(a, dtype):
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.ascontiguousarray(a, np.float64)).float().to(dtype)


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def forward(z, F, act):
    """(h, its error) in float64."""
    g = z[:, :F]
    with np.errstate(invalid="ignore"):
        s = g * sigmoid(g)
        h = s * z[:, F:] if act == "swiglu" else s
        return h, (2 * np.abs(g) + 9) * U * np.abs(h)


def backward(da, z, F, act):
    """(dz, its error)."""
    g = z[:, :F]
    s = sigmoid(g)
    a = g * s
    slope, dslope = s + a * (1 - s), (2 * np.abs(g) + 10) * U * (s + 2 * np.abs(a))
    if act == "silu":
        return da * slope, np.abs(da) * dslope + 2 * U * np.abs(da * slope)
    u = z[:, F:]
    dz = np.concatenate([da * u * slope, da * a], 1)
    return dz, np.concatenate([np.abs(da * u) * dslope + 3 * U * np.abs(da * u * slope),
                               (2 * np.abs(g) + 10) * U * np.abs(da * a)], 1)


def check_quantized(got, want, error, dtype, fmt, dim):
    """`got` (data, scale) against the quantize of `want` rounded to dtype, each value off by
    at most `error` before that."""
    data, scale = (t.cpu().numpy() for t in got)
    def quantized(a):
        d, s = oracle.quantize_axis(bits(rounded(a, dtype)), NAMES[dtype], fmt, dim, layout="dense")
        return d, s

    d, s = quantized(want)
    assert data.shape == d.shape and scale.shape == s.shape
    K, O = 32 * s.shape[0], s.shape[1]

    def same(a, b):
        """[K/32, O]: blocks of equal codes (zeros of either sign) and scales."""
        zero = 0x80 if fmt != "e2m1" else 8
        x, y = (t[0] if fmt != "e2m1" else np.stack([t[0] & 15, t[0] >> 4], -1) for t in (a, b))
        x, y = (np.where(t == zero, 0, t).reshape(K // 4, O, -1) for t in (x, y))
        return (x == y).all(2).reshape(K // 32, 8, O).all(1) & (a[1] == b[1])

    nan = np.isnan(want)
    sure = same(quantized(np.where(nan, want, want - error)), quantized(np.where(nan, want, want + error)))
    assert sure.mean() > 0.5      # the comparison here is the rule, the one below the exception
    assert same((data, scale), (d, s))[sure].all()
    # the others
    v = values(data, scale, fmt)
    w = want.T if dim == -1 else want
    err = error.T if dim == -1 else error
    half, emax, largest = FORMAT[fmt]
    assert (np.abs(scale.astype(int) - s) <= 1).all()
    unit = np.repeat(np.ldexp(1.0, scale.astype(np.int64) - 127), 32, axis=0)
    # (a value past the largest code gives that one)
    allowed = half * 2.0 ** emax * unit + err + 2 * np.abs(w) * float(torch.finfo(dtype).eps) + 2.0 ** -24
    off = np.abs(v - np.clip(w, -largest * unit, largest * unit))
    unsure = np.repeat(~sure, 32, axis=0) & np.isfinite(w)
    assert (off <= allowed)[unsure].all()


def inputs(R, F, act, dtype, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    W = 2 * F if act == "swiglu" else F
    return (torch.randn((R, W), generator=g) * scale).to(dtype), (torch.randn((R, F), generator=g) * 1e-2).to(dtype)


def check_forward(z, F, act, out, saved):
    progress("act %s %s %s to %s, kept %s" % (tuple(z.shape), act, z.dtype, out, saved))
    got, kept = mxq.act_quantize(z.cuda(), act, out, saved)
    d, s = oracle.quantize(bits(z), NAMES[z.dtype], saved, layout="dense")
    assert np.array_equal(kept[0].cpu().numpy(), d) and np.array_equal(kept[1].cpu().numpy(), s)
    h, error = forward(z.double().numpy(), F, act)
    check_quantized(got, h, error, z.dtype, out, -1)


def check_backward(z, da, F, act, out, saved, patch=None):
    progress("act backward %s %s %s to %s, kept %s" % (tuple(da.shape), act, da.dtype, out, saved))
    R, W = z.shape
    d, s = oracle.quantize(bits(z), NAMES[z.dtype], saved, layout="dense")
    if patch:
        patch(d, s)
    got = mxq.act_quantize_backward(da.cuda(), dev(d), dev(s), act, saved, out)
    kept = oracle.dequantize(d, s, R, W, saved, layout="dense").astype(np.float64)
    with np.errstate(all="ignore"):
        h, herr = forward(kept, F, act)
        dz, derr = backward(da.double().numpy(), kept, F, act)
    check_quantized(got.rows, dz, derr, da.dtype, out, -1)
    check_quantized(got.cols, dz, derr, da.dtype, out, -2)
    check_quantized(got.h, h, herr, da.dtype, out, -2)


@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out", ["e4m3fn", "e5m2", "e2m1"])
@pytest.mark.parametrize("saved", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("R,F", [(8, 32), (40, 96), (32, 128), (64, 160), (296, 1056)])
def test_forward(R, F, saved, out, dtype, act):
    z, _ = inputs(R, F, act, dtype, R + F)
    check_forward(z, F, act, out, saved)


@pytest.mark.parametrize("act", ["swiglu", "silu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out", ["e4m3fn", "e5m2", "e2m1"])
@pytest.mark.parametrize("saved", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("R,F", [(32, 32), (64, 96), (32, 128), (96, 160), (288, 1056)])
def test_backward(R, F, saved, out, dtype, act):
    z, da = inputs(R, F, act, dtype, R + F)
    check_backward(z, da, F, act, out, saved)


@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_large_arguments(act):
    """Far into both tails, where the exponential overflows or vanishes."""
    z, da = inputs(64, 64, act, torch.bfloat16, 7, scale=60.0)
    check_forward(z, 64, act, "e4m3fn", "e4m3fn")
    check_backward(z, da, 64, act, "e4m3fn", "e5m2")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out", ["e4m3fn", "e5m2", "e2m1"])
def test_infinities_and_nan(dtype, out):
    """A NaN is kept and quantized as a zero of its sign, an infinity as the largest value;
    blocks without either are as they would be."""
    F = 96
    z, da = inputs(64, F, "swiglu", dtype, 11)
    want = mxq.act_quantize(z.cuda(), "swiglu", out)
    bad = z.clone()
    bad[3, 5], bad[17, F + 40], bad[40, 70], bad[41, F + 70] = float("nan"), float("inf"), float("inf"), float("nan")
    (d, s), (k, ks) = mxq.act_quantize(bad.cuda(), "swiglu", out)
    kd, kss = oracle.quantize(bits(bad), NAMES[dtype], "e4m3fn", layout="dense")
    assert np.array_equal(k.cpu().numpy(), kd) and np.array_equal(ks.cpu().numpy(), kss)
    v = values(d.cpu().numpy(), s.cpu().numpy(), out)      # [F, R]
    assert np.isfinite(v).all() and v[5, 3] == 0 and v[70, 41] == 0
    w = values(*(t.cpu().numpy() for t in want[0]), out)
    touched = np.zeros((F, 64), bool)
    for r, c in ((3, 5), (17, 40), (40, 70), (41, 70)):
        touched[c // 32 * 32:c // 32 * 32 + 32, r] = True
    assert np.array_equal(v[~touched], w[~touched])
    assert abs(v[40, 17]) > 2.0 ** 100 if dtype == torch.bfloat16 else abs(v[40, 17]) > 2.0 ** 15

    da[9, 33] = float("nan")
    da[50, 2] = float("inf")
    want = mxq.act_quantize(z.cuda(), "swiglu", out)[1]
    got = mxq.act_quantize_backward(da.cuda(), *want, "swiglu", "e4m3fn", out)
    rows = values(*(t.cpu().numpy() for t in got.rows), out)     # [2 F, R]
    cols = values(*(t.cpu().numpy() for t in got.cols), out)     # [R, 2 F]
    for a in (rows.T, cols):
        assert np.isfinite(a).all() and a[9, 33] == 0 and a[9, F + 33] == 0


@pytest.mark.parametrize("act", ["swiglu", "silu"])
def test_kept_scale_bytes_at_their_ends(act):
    """Scale bytes 0 (2^-127) and 255 (2^128) of the kept input have their values."""
    def patch(d, s):
        s[0, :3] = 0
        s[2, 1] = 0
        d[8:16, 0:4] = 0x38      # 1.0 in e4m3
        s[1, 0] = 0
        d[16:24, 4:8] = np.where(np.arange(4) % 2, 0x01, 0x81)   # +- 2^-9, times 2^128: gates of +- 2^119
        s[2, 1] = 255

    z, da = inputs(64, 64, act, torch.bfloat16, 13)
    check_backward(z, da, 64, act, "e4m3fn", "e4m3fn", patch)


def test_gradient_against_differences():
    """dz is the slope of sum(da * h): central differences in 64 bits at the decoded z."""
    F, R = 32, 32
    z, da = inputs(R, F, "swiglu", torch.bfloat16, 17)
    kept = mxq.act_quantize(z.cuda(), "swiglu")[1]
    zk = mxq.dequantize(*kept, "e4m3fn", torch.float32, dense_scale=True).double().cpu().numpy()
    got = values(*(t.cpu().numpy() for t in mxq.act_quantize_backward(da.cuda(), *kept).rows), "e4m3fn").T
    scale = np.abs(got).reshape(R, 2 * F // 32, 32).max(2)
    step = 1e-5
    for r in range(0, R, 7):
        for c in range(2 * F):
            p, m = zk[r:r + 1].copy(), zk[r:r + 1].copy()
            p[0, c] += step
            m[0, c] -= step
            d = ((forward(p, F, "swiglu")[0] - forward(m, F, "swiglu")[0]) * da[r].double().numpy()).sum() / (2 * step)
            # half a step of e4m3 at the block's largest value, and of bf16
            assert abs(got[r, c] - d) <= 2.0 ** -4 * 2 * scale[r, c // 32] + 2.0 ** -8 * abs(d) + 1e-8


def test_rows_do_not_depend_on_each_other():
    """A call on some rows gives those rows' bytes, whatever the tile they lie in."""
    z, _ = inputs(200, 416, "swiglu", torch.bfloat16, 19)
    (d, s), (k, ks) = mxq.act_quantize(z.cuda(), "swiglu")
    for a, b in ((0, 8), (8, 56), (104, 200)):
        (d2, s2), (k2, ks2) = mxq.act_quantize(z[a:b].contiguous().cuda(), "swiglu")
        assert torch.equal(d.view(104, 200, 4)[:, a:b], d2.view(104, b - a, 4)) and torch.equal(s[:, a:b], s2)
        assert torch.equal(k[a:b], k2) and torch.equal(ks[a // 8:b // 8], ks2)


def test_empty():
    for shape in ((0, 64), (8, 0)):
        (d, s), (k, ks) = mxq.act_quantize(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), "silu")
        assert d.numel() == s.numel() == k.numel() == ks.numel() == 0
    z = torch.zeros((0, 32), dtype=torch.bfloat16, device="cuda")
    u8 = torch.zeros((0, 32), dtype=torch.uint8, device="cuda")
    assert mxq.act_quantize_backward(z, u8, u8[:, :8].contiguous(), "silu").h[0].numel() == 0


def test_other_stream_graph_and_repeats():
    z, da = (t.cuda() for t in inputs(288, 416, "swiglu", torch.bfloat16, 23))

    def run(**kw):
        out, kept = mxq.act_quantize(z, "swiglu", **kw)
        return (*out, *kept, *sum(mxq.act_quantize_backward(da, *kept, **kw), ()))

    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got, here = run(stream=s), run()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got + here, want + want))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for _ in range(4):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        _ = (da.float() * 2).sum().item()
