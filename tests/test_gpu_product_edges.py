"""GPU tests of the products where a wave's part of a tile lies past the result's last
row or column while the operands hold scale bytes of 255 or NaN codes: such a part
takes no second pass and changes no result. Bounds as in test_gpu_grouped."""
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_grouped import check_rows, compare, dev, host, quantized, values
from test_gpu_grouped_forms import check_wgrad

pytestmark = pytest.mark.gpu


def scales(l, ls, r, rs):
    """255 in the last block's last columns, small scales on the other side."""
    ls[-1, -3:] = 255
    ls[-1, :-3] = 100
    rs[..., -1, -1] = 255
    rs[..., -1, :-1] = 24


def codes(l, ls, r, rs):
    l[-1, -1] = 0x7F
    r[..., -1, -4] = 0xFF


# widths whose last 256-column tile has less than 128 columns, and rows whose last
# tile has 64 or less; 4 by 4: the operand is shorter than a wave's start column
@pytest.mark.parametrize("patch", [scales, codes])
@pytest.mark.parametrize("sizes,M,N", [([32, 64], 4, 4), ([64], 4, 300), ([32, 0, 64], 260, 4), ([800], 300, 260),
                                       ([1536], 4, 4)])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_wgrad(sizes, M, N, res, patch):
    progress("grouped wgrad %s M=%d N=%d %s %s" % (sizes, M, N, res, patch.__name__))
    check_wgrad(sizes, M, N, "e4m3fn", res, 41, patch, per_block=4)


@pytest.mark.parametrize("patch", [scales, codes])
@pytest.mark.parametrize("sizes,K,N", [([132, 68, 260], 96, 2564), ([500, 700, 604], 96, 2600),
                                       ([500, 700, 604], 1056, 2600), ([32] * 3, 64, 4)])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_rows(sizes, K, N, res, patch):
    progress("grouped rows %s K=%d N=%d %s %s" % (sizes, K, N, res, patch.__name__))
    check_rows(sizes, 0, K, N, "e4m3fn", res, seed=43, patch=patch, per_block=4)


@pytest.mark.parametrize("patch", [scales, codes])
@pytest.mark.parametrize("M,N", [(4, 4), (300, 260), (4, 300), (516, 292)])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
def test_scaled_matmul(M, N, res, patch):
    progress("scaled matmul M=%d N=%d %s %s" % (M, N, res, patch.__name__))
    l, ls = quantized(160, M, -2, "e4m3fn", M)
    r, rs = quantized(160, N, -2, "e4m3fn", N + 1)
    patch(l, ls, r, rs)
    big = torch.full((M * N + 64,), 7.0, dtype=res, device="cuda")
    mxq.scaled_matmul(dev(l), dev(ls), dev(r), dev(rs), "e4m3fn", res, out=big[:M * N].view(M, N), dense_scale=True)
    got = host(big)
    assert (got[M * N:] == 7).all()
    compare(got[:M * N].reshape(M, N), values(l, ls, "e4m3fn"), values(r, rs, "e4m3fn"), res, 4)
