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
