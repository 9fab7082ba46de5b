"""Refusals and size queries of the mixture-of-experts and clipping calls: every
one is made before anything is launched, so no GPU is needed."""
import ctypes

import numpy as np
import pytest
import torch

import moe_reference as ref
import mx_microscaling_quantization_amd as mxq

E_IN, E_OUT, E_P8, E_F4, E_NULL, E_ALIGN, E_OVERFLOW, E_FLAGS, E_RES, E_DIM = 1, 2, 3, 4, 5, 6, 7, 9, 10, 11
E_MOE, E_ROWS, E_ELEM, E_VALUE = 12, 13, 14, 15
OK = 0
GOOD = 4096   # an aligned address that no refused call reads


@pytest.mark.parametrize("T,k,E,align", [(0, 1, 1, 32), (1, 8, 8, 32), (1, 8, 256, 32), (61, 4, 32, 4), (1000, 6, 64, 128),
                                         (65536, 8, 256, 32), (5, 64, 1024, 256)])
def test_rows(T, k, E, align):
    assert mxq.moe_rows(T, k, E, align) == ref.rows_needed(T * k, E, align)


@pytest.mark.parametrize("seed", range(5))
def test_rows_hold_any_assignment(seed):
    g = np.random.default_rng(seed)
    T, k, E, align = int(g.integers(1, 60)), int(g.integers(1, 9)), int(g.integers(1, 40)), int(4 * g.integers(1, 17))
    for hi in (1, E):   # all to one expert, spread over all
        ids = g.integers(0, hi, size=(T, k))
        offsets, src, _ = ref.sort(ids, E, align)
        assert offsets[-1] <= src.size == mxq.moe_rows(T, k, E, align)


@pytest.mark.parametrize("args", [(-1, 1, 8, 32), (4, 0, 8, 32), (4, 65, 8, 32), (4, 2, 0, 32), (4, 2, 1025, 32),
                                  (4, 2, 8, 0), (4, 2, 8, 6), (4, 2, 8, 260), (1 << 31, 2, 8, 32)])
def test_rows_refused(args):
    assert mxq.load().mxq_moe_rows(*args) == -1
    with pytest.raises(mxq.MXQError):
        mxq.moe_rows(*args)


def test_sort_refusals():
    f = mxq.load().mxq_moe_sort
    g = GOOD

    def call(ids=g, nb=4, T=16, k=2, E=8, align=32, off=g, src=g, dest=g, ws=g):
        return f(ids, nb, T, k, E, align, off, src, dest, ws, None)

    assert call(nb=2) == E_ELEM
    assert call(T=-1) == E_MOE and call(k=0) == E_MOE and call(k=65) == E_MOE
    assert call(E=0) == E_MOE and call(E=1025) == E_MOE
    assert call(align=2) == E_MOE and call(align=34) == E_MOE and call(align=512) == E_MOE
    assert call(T=1 << 40) == E_OVERFLOW
    for name in ("ids", "off", "src", "dest"):
        assert call(**{name: None}) == E_NULL, name
        assert call(**{name: g + 4}) == E_ALIGN, name
    assert call(T=1 << 20, ws=None) == E_NULL
    assert mxq.load().mxq_moe_sort_workspace_bytes(1 << 20, 2, 8) > 0
    assert mxq.load().mxq_moe_sort_workspace_bytes(16, 2, 8) == 0


def test_gather_quantize_refusals():
    f = mxq.load().mxq_moe_gather_quantize
    g = GOOD

    def call(x=g, T=4, k=2, K=64, it=0, ot=0, dim=-1, flags=2, src=g, rows=32, d=g, s=g):
        return f(x, T, k, K, it, ot, dim, flags, src, rows, d, s, None)

    assert call(it=2) == E_IN and call(ot=3) == E_OUT and call(flags=4) == E_FLAGS
    assert call(dim=2) == E_DIM and call(dim=-3) == E_DIM
    assert call(k=0) == E_MOE and call(T=-1) == E_MOE
    assert call(rows=-4) == E_ROWS and call(rows=30) == E_ROWS
    assert call(T=0) == E_ROWS
    assert call(K=48) == E_P8 and call(dim=-2, rows=36) == E_P8 and call(K=-32) == E_F4
    assert call(rows=1 << 40) == E_OVERFLOW
    assert call(rows=0) == OK and call(K=0) == OK
    for name in ("x", "src", "d", "s"):
        assert call(**{name: None}) == E_NULL, name
        assert call(**{name: g + 8}) == E_ALIGN, name


def test_combine_refusals():
    lib, g = mxq.load(), GOOD

    def fwd(y=g, rows=32, N=64, et=0, dest=g, w=g, T=4, k=2, out=g):
        return lib.mxq_moe_combine(y, rows, N, et, dest, w, T, k, out, None)

    def bwd(grad=g, y=g, rows=32, N=64, et=0, src=g, dest=g, w=g, T=4, k=2, gy=g, gw=g):
        return lib.mxq_moe_combine_backward(grad, y, rows, N, et, src, dest, w, T, k, gy, gw, None)

    for call in (fwd, bwd):
        assert call(et=3) == E_ELEM and call(et=-1) == E_ELEM
        assert call(k=0) == E_MOE and call(k=65) == E_MOE and call(T=-1) == E_MOE
        assert call(rows=-1) == E_ROWS and call(N=-1) == E_ROWS
        assert call(rows=1 << 33) == E_OVERFLOW and call(N=1 << 33) == E_OVERFLOW
    assert fwd(T=1 << 20, N=1 << 20) == E_OVERFLOW          # more work-items than a dispatch counts
    assert fwd(T=0) == OK and fwd(N=0) == OK
    assert bwd(T=0, rows=0) == OK
    for name in ("y", "dest", "out"):
        assert fwd(**{name: None}) == E_NULL and fwd(**{name: g + 2}) == E_ALIGN, name
    assert fwd(w=g + 4) == E_ALIGN
    for name in ("grad", "y", "src", "dest", "w", "gy", "gw"):
        assert bwd(**{name: None}) == E_NULL and bwd(**{name: g + 4}) == E_ALIGN, name


@pytest.mark.parametrize("wgrad", [False, True])
def test_grouped_matmul_refusals(wgrad):
    lib, g = mxq.load(), GOOD
    f = lib.mxq_grouped_matmul_wgrad if wgrad else lib.mxq_grouped_matmul

    def call(l=g, ls=g, r=g, rs=g, off=g, G=4, P=16, M=64, N=64, fmt=0, res=1, out=g):
        return f(l, ls, r, rs, off, G, P, M, N, fmt, res, out, None)

    assert call(fmt=2) == E_OUT and call(fmt=-1) == E_OUT and call(res=2) == E_RES
    assert call(G=0) == E_MOE and call(G=1025) == E_MOE
    assert call(P=12) == E_P8 and call(P=-8) == E_P8
    assert call(M=62) == E_F4 and call(N=66) == E_F4 and call(M=-4) == E_F4
    assert call(M=33554180) == E_OVERFLOW and call(N=33554180) == E_OVERFLOW and call(P=1 << 30) == E_OVERFLOW
    assert call(M=33554176, N=33554176) == E_OVERFLOW
    assert call(M=0) == OK and call(N=0) == OK
    for name in ("l", "ls", "r", "rs", "off", "out"):
        assert call(**{name: None}) == E_NULL, name
        assert call(**{name: g + 4}) == E_ALIGN, name


def _clip(ptrs, outs, numels, codes, max_norm=1.0, norm=GOOD, ws=GOOD):
    n = len(ptrs)
    P = ctypes.c_void_p * n
    return mxq.load().mxq_clip_grad_norm(P(*ptrs), None if outs is None else P(*outs), (ctypes.c_int64 * n)(*numels),
                                         (ctypes.c_int * n)(*codes), n, max_norm, norm, ws, None)


def test_clip_refusals():
    g = GOOD
    assert _clip([g], [g], [4], [3]) == E_ELEM
    assert _clip([g], [g], [-1], [0]) == E_ROWS
    assert _clip([g], [g], [1 << 41], [0]) == E_OVERFLOW
    assert _clip([g], [g], [4], [0], max_norm=-1.0) == E_VALUE
    assert _clip([g], [g], [4], [0], max_norm=float("nan")) == E_VALUE
    assert _clip([None], [g], [4], [0]) == E_NULL and _clip([g], [None], [4], [0]) == E_NULL
    assert _clip([g], [g], [4], [0], norm=None) == E_NULL and _clip([g], [g], [4], [0], ws=None) == E_NULL
    assert _clip([g + 1], [g], [4], [0]) == E_ALIGN and _clip([g + 2], [g], [4], [2]) == E_ALIGN
    assert _clip([g], [g + 2], [4], [2]) == E_ALIGN and _clip([g], [g], [4], [0], ws=g + 8) == E_ALIGN
    f = mxq.load().mxq_clip_grad_norm_workspace_bytes
    assert f((ctypes.c_int64 * 1)(4), (ctypes.c_int * 1)(7), 1) == 0
    assert f((ctypes.c_int64 * 1)(4), (ctypes.c_int * 1)(0), 1) >= 8
    with pytest.raises(mxq.MXQError):
        mxq.clip_grad_norm([], -1.0)
    with pytest.raises(ValueError):
        mxq.clip_grad_norm([], 1.0)


def test_binding_refuses_host_tensors_and_wrong_types():
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        mxq.moe_sort(ids, 4)
    plan = mxq.MoEPlan(torch.zeros(5, dtype=torch.int32), torch.zeros(32, dtype=torch.int32), ids)
    with pytest.raises(ValueError):
        mxq.moe_gather_quantize(torch.zeros((4, 32), dtype=torch.bfloat16), plan)
    with pytest.raises(mxq.MXQError):
        mxq.moe_gather_quantize(torch.zeros((4, 32)), plan)
    with pytest.raises(mxq.MXQError):
        mxq.moe_combine(torch.zeros((32, 8), dtype=torch.float64), plan)
    with pytest.raises(ValueError):
        mxq.moe_combine(torch.zeros((32, 8)), plan)
    with pytest.raises(ValueError):
        mxq.clip_grad_norm([torch.zeros(4)], 1.0)
    u8 = torch.zeros((8, 16), dtype=torch.uint8)
    with pytest.raises(ValueError):
        mxq.grouped_scaled_matmul(u8, u8, u8, u8, ids)
    with pytest.raises(mxq.MXQError):
        mxq.grouped_scaled_matmul(u8, u8, u8, u8, ids, "e4m3fn", torch.float16)
    with pytest.raises(ValueError):
        mxq.grouped_scaled_matmul_wgrad(u8, u8, u8, u8, ids)


# The references' own pins.

def test_reference_sort_by_hand():
    ids = np.array([[2, 0], [0, 7], [2, -1], [2, 0]])
    offsets, src, dest = ref.sort(ids, 3, 4)
    assert offsets.tolist() == [0, 4, 4, 8]
    assert src.tolist() == [1, 2, 7, -1, 0, 4, 6, -1] + [-1] * 8
    assert dest.tolist() == [[4, 0], [1, -1], [5, -1], [6, 2]]


def test_reference_gradient_against_differences():
    g = np.random.default_rng(1)
    ids = g.integers(0, 5, size=(6, 3))
    _, src, dest = ref.sort(ids, 4, 4)
    y, w, grad = g.normal(size=(src.size, 5)), g.normal(size=(6, 3)), g.normal(size=(6, 5))
    gy, gw, _ = ref.combine_backward(grad, y, src, dest, w)
    h = 1e-3
    for t, j in [(0, 0), (3, 2), (5, 1)]:
        p, m = w.copy(), w.copy()
        p[t, j] += h
        m[t, j] -= h
        d = ((ref.combine(y, dest, p)[0] - ref.combine(y, dest, m)[0]) * grad).sum() / (2 * h)
        assert abs(d - gw[t, j]) < 1e-9
    for r, n in [(0, 0), (int(dest.max()), 4)]:
        p, m = y.copy(), y.copy()
        p[r, n] += h
        m[r, n] -= h
        d = ((ref.combine(p, dest, w)[0] - ref.combine(m, dest, w)[0]) * grad).sum() / (2 * h)
        assert abs(d - gy[r, n]) < 1e-9
