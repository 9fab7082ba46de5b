"""GPU tests of the calls around the experts at lists and plans that the other tests
leave out. Bounds as in test_gpu_moe."""
import numpy as np
import pytest
import torch

import moe_reference as ref
import mx_microscaling_quantization_amd as mxq
from conftest import progress
from test_gpu_moe import host, make_ids, plan_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [3, 64, 600, 4096])
def test_gradient_of_pairs_taken_out_of_dest_alone(N):
    """dest without some pairs, src as it was: their weights have a zero gradient, the
    others' is the dot product, every time."""
    T, k, E = 40, 3, 5
    progress("combine gradient, dest changed alone, N=%d" % N)
    plan = plan_of(make_ids(T, k, E, 11), E)
    rows = plan.src.numel()
    g = torch.Generator().manual_seed(N)
    y, w = torch.randn((rows, N), generator=g).cuda(), torch.rand((T, k), generator=g).cuda()
    grad = torch.randn((T, N), generator=g).cuda()
    dest = plan.dest.clone()
    dest[::2, 1] = -1
    dest[1::4, 0] = dest[0, 0]      # another pair's row
    changed = mxq.MoEPlan(plan.offsets, plan.src, dest)
    named = (dest >= 0) & (dest == plan.dest)
    want, _, _ = ref.combine_backward(host(grad), host(y), plan.src.cpu().numpy(), plan.dest.cpu().numpy(), host(w))
    _, dots, mags = ref.combine_backward(host(grad), host(y), plan.src.cpu().numpy(), dest.cpu().numpy(), host(w))
    for _ in range(5):
        gy, gw = mxq.moe_combine_backward(grad, y, changed, w, grad_weights=torch.full((T, k), 9.0, device="cuda"))
        assert bool((gw[~named] == 0).all())
        off = np.abs(host(gw) - dots) <= (N + 8) * 2.0 ** -24 * mags
        assert off[named.cpu().numpy()].all()
        assert (np.abs(host(gy) - want) <= 2.0 ** -24 * np.abs(want)).all()


# One workgroup sorts up to 4096 pairs, each wave at most the 4 x 64 whose numbers it
# keeps in registers; 4097 pairs are three chunks of 2048, the last with one pair.
# 524288 pairs are the most in chunks of 2048 or 4096, 2^20 in 256 chunks of 4096.
@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("T,k,E,align", [(4095, 1, 64, 32), (4096, 1, 64, 32), (4097, 1, 64, 32), (512, 8, 128, 32),
                                         (513, 8, 128, 32), (1365, 3, 1024, 4), (1366, 3, 1024, 4), (6144, 1, 5, 256),
                                         (6145, 1, 5, 256), (65536, 8, 16, 32), (65537, 8, 256, 32), (131072, 8, 33, 32),
                                         (131073, 8, 33, 32)])
def test_sort_about_its_limits(T, k, E, align, dtype):
    progress("sort T=%d k=%d E=%d align=%d %s" % (T, k, E, align, dtype.__name__))
    ids = make_ids(T, k, E, seed=T + E, dtype=dtype)
    for got, want in zip(plan_of(ids, E, align), ref.sort(ids, E, align)):
        assert np.array_equal(got.cpu().numpy(), want)
