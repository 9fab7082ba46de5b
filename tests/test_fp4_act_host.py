"""Refusals and size queries of the products with 4-bit weights, the layer for a few
tokens and the activations between products: every one is made before anything is
launched, so no GPU is needed."""
import pytest
import torch

import mx_microscaling_quantization_amd as mxq

E_IN, E_OUT, E_P8, E_F4, E_NULL, E_ALIGN, E_OVERFLOW, E_FLAGS, E_RES = 1, 2, 3, 4, 5, 6, 7, 9, 10
E_MOE, E_ROWS, E_ELEM, E_ACT = 12, 13, 14, 16
OK = 0
GOOD = 4096   # an aligned address that no refused call reads
E2M1 = mxq.OUT_DTYPES["e2m1"]


def dense(l=GOOD, ls=GOOD, r=GOOD, rs=GOOD, P=8, M=4, N=4, fmt=0, res=0, flags=0, out=GOOD):
    return mxq.load().mxq_scaled_matmul_fp4(l, ls, r, rs, P, M, N, fmt, res, flags, out, None)


def grouped(l=GOOD, ls=GOOD, r=GOOD, rs=GOOD, off=GOOD, G=2, P=8, rows=4, N=4, fmt=0, res=0, out=GOOD):
    return mxq.load().mxq_grouped_matmul_fp4(l, ls, r, rs, off, G, P, rows, N, fmt, res, out, None)


def few(x=GOOD, T=4, K=32, dt=0, ids=GOOD, nb=4, w=GOOD, k=2, E=8, w1=GOOD, w1s=GOOD, w2=GOOD, w2s=GOOD, F=32, N=4,
        fmt=0, act=1, ws=GOOD, out=GOOD):
    return mxq.load().mxq_moe_few_tokens(x, T, K, dt, ids, nb, w, k, E, w1, w1s, w2, w2s, F, N, fmt, act, ws, out,
                                         None)


def act(z=GOOD, R=32, F=32, dt=0, out=0, saved=0, act=1, d=GOOD, s=GOOD, k=GOOD, ks=GOOD):
    return mxq.load().mxq_act_quantize(z, R, F, dt, out, saved, act, d, s, k, ks, None)


def back(g=GOOD, k=GOOD, ks=GOOD, R=32, F=32, dt=0, out=0, saved=0, act=1, rd=GOOD, rs=GOOD, cd=GOOD, cs=GOOD,
         hd=GOOD, hs=GOOD):
    return mxq.load().mxq_act_quantize_backward(g, k, ks, R, F, dt, out, saved, act, rd, rs, cd, cs, hd, hs, None)


@pytest.mark.parametrize("call", [dense, grouped])
def test_fp4_refusals(call):
    rows = "M" if call is dense else "rows"
    assert call(fmt=3) == E_OUT and call(fmt=-1) == E_OUT
    assert call(res=2) == E_RES and call(res=-1) == E_RES
    assert call(P=4) == E_P8 and call(P=-8) == E_P8
    assert call(N=6) == E_F4 and call(N=-4) == E_F4
    assert call(P=1 << 29) == E_OVERFLOW and call(N=33554176 + 4) == E_OVERFLOW
    assert call(**{rows: 33554176 + 4}) == E_OVERFLOW
    for name in ("l", "ls", "r", "rs", "out"):
        assert call(**{name: None}) == E_NULL, name
        assert call(**{name: GOOD + 8}) == E_ALIGN, name
    assert call(N=0) == OK and call(**{rows: 0}) == OK
    # more tiles than a grid holds
    assert call(**{rows: 33554176, "N": 33554176}) == E_OVERFLOW


def test_fp4_own_refusals():
    assert dense(M=-1) == E_F4 and dense(flags=1) == E_FLAGS and dense(flags=2 | 4) == E_FLAGS
    assert grouped(rows=6) == E_ROWS and grouped(rows=-4) == E_ROWS
    assert grouped(G=0) == E_MOE and grouped(G=1025) == E_MOE
    assert grouped(off=None) == E_NULL and grouped(off=GOOD + 4) == E_ALIGN


def test_few_tokens_refusals():
    assert few(dt=2) == E_IN and few(fmt=3) == E_OUT and few(act=2) == E_ACT and few(act=-1) == E_ACT
    assert few(nb=2) == E_ELEM
    assert few(T=-1) == E_MOE and few(k=0) == E_MOE and few(k=65) == E_MOE
    assert few(E=0) == E_MOE and few(E=1025) == E_MOE
    assert few(T=513) == E_MOE and few(T=1 << 60, k=64) == E_MOE     # more than 1024 pairs
    assert few(K=16) == E_P8 and few(F=48) == E_P8 and few(K=-32) == E_P8 and few(F=-32) == E_P8
    assert few(N=6) == E_F4 and few(N=-4) == E_F4
    assert few(K=1 << 31) == E_OVERFLOW and few(N=1 << 31) == E_OVERFLOW
    assert few(K=1 << 20, F=1 << 10) == E_OVERFLOW and few(F=1 << 20, N=1 << 11) == E_OVERFLOW
    for name in ("x", "ids", "w", "w1", "w1s", "w2", "w2s", "ws", "out"):
        assert few(**{name: None}) == E_NULL, name
        assert few(**{name: GOOD + 4}) == E_ALIGN, name
    assert few(T=0) == OK and few(N=0) == OK


def test_few_tokens_workspace():
    size = mxq.load().mxq_moe_few_tokens_workspace_bytes
    # both halves of h, y, and 8-column tiles' counters fit
    assert size(16, 4, 2048, 4096) >= 16 * 4 * 4 * (2048 + 4096)
    assert size(513, 2, 32, 4) == 0 and size(4, 0, 32, 4) == 0 and size(4, 2, 33, 4) == 0
    assert size(-1, 2, 32, 4) == 0 and size(4, 2, 32, 5) == 0


def test_act_refusals():
    for call in (act, back):
        assert call(dt=2) == E_IN and call(out=3) == E_OUT and call(saved=E2M1) == E_OUT and call(saved=7) == E_OUT
        assert call(act=2) == E_ACT and call(act=-1) == E_ACT
        assert call(R=-32) == E_P8 and call(F=-32) == E_P8 and call(F=16) == E_P8 and call(R=4) == E_P8
        assert call(R=1 << 31) == E_OVERFLOW and call(F=1 << 30) == E_OVERFLOW
        assert call(R=1 << 30, F=1 << 29) == E_OVERFLOW      # more tiles than a grid holds
        assert call(R=0) == OK and call(F=0) == OK
    assert back(R=8) == E_P8                 # blocks down the columns are of 32 rows
    for name in ("z", "d", "s", "k", "ks"):
        assert act(**{name: None}) == E_NULL and act(**{name: GOOD + 8}) == E_ALIGN, name
    for name in ("g", "k", "ks", "rd", "rs", "cd", "cs", "hd", "hs"):
        assert back(**{name: None}) == E_NULL and back(**{name: GOOD + 8}) == E_ALIGN, name


def test_status_string():
    assert "activation" in mxq.status_string(E_ACT).lower()


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_bindings_refuse_host_tensors_and_wrong_types():
    with pytest.raises(ValueError):
        mxq.scaled_matmul_fp4(u8(8, 16), u8(1, 4), u8(8, 8), u8(1, 4), dense_scale=True)
    with pytest.raises(ValueError):
        mxq.grouped_scaled_matmul_fp4(u8(8, 16), u8(1, 4), u8(2, 8, 8), u8(2, 1, 4), torch.zeros(3, dtype=torch.int32))
    for call in (mxq.scaled_matmul_fp4,):
        with pytest.raises(mxq.MXQError):
            call(u8(8, 16), u8(1, 4), u8(8, 8), u8(1, 4), "e3m2")
        with pytest.raises(mxq.MXQError):
            call(u8(8, 16), u8(1, 4), u8(8, 8), u8(1, 4), "e4m3fn", torch.float16)
    bf = torch.zeros((4, 32), dtype=torch.bfloat16)
    layer = (torch.zeros((4, 2), dtype=torch.int64), torch.zeros((4, 2)), u8(2, 8, 128), u8(2, 1, 64), u8(2, 8, 8),
             u8(2, 1, 4))
    with pytest.raises(ValueError):
        mxq.moe_few_tokens(bf, *layer)
    with pytest.raises(mxq.MXQError):
        mxq.moe_few_tokens(bf.float(), *layer)
    with pytest.raises(mxq.MXQError):
        mxq.moe_few_tokens(bf, *layer, fmt="e3m2")
    with pytest.raises(mxq.MXQError):
        mxq.moe_few_tokens(bf, *layer, activation="gelu")
    with pytest.raises(ValueError):
        mxq.act_quantize(torch.zeros((32, 64), dtype=torch.bfloat16))
    with pytest.raises(mxq.MXQError):
        mxq.act_quantize(torch.zeros((32, 64)))
    with pytest.raises(mxq.MXQError):
        mxq.act_quantize(bf, "relu")
    with pytest.raises(mxq.MXQError):
        mxq.act_quantize(bf, saved_dtype="e2m1")
    with pytest.raises(ValueError):
        mxq.act_quantize_backward(torch.zeros((32, 32), dtype=torch.bfloat16), u8(32, 64), u8(4, 16))
    with pytest.raises(mxq.MXQError):
        mxq.act_quantize_backward(torch.zeros((32, 32)), u8(32, 64), u8(4, 16))
    with pytest.raises(mxq.MXQError):
        mxq.act_quantize_backward(torch.zeros((32, 32), dtype=torch.bfloat16), u8(32, 64), u8(4, 16), out_dtype="e8m0")
