"""GPU tests of what autograd sees of the calls: tensors that a call writes to count a
new version, so a backward pass that kept one from before refuses to run."""
import pytest
import torch

import mx_microscaling_quantization_amd as mxq
from test_gpu_moe import make_ids, plan_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("to_out", [False, True])
def test_clipped_tensors_count_a_version(to_out):
    grads = [torch.ones(100, device="cuda"), torch.ones((3, 5), device="cuda", dtype=torch.bfloat16),
             torch.zeros(0, device="cuda")]
    outs = [torch.empty_like(g) for g in grads]
    before = [(g._version, o._version) for g, o in zip(grads, outs)]
    mxq.clip_grad_norm(grads, 0.5, out=outs if to_out else None)
    for (g0, o0), g, o in zip(before, grads, outs):
        assert (g._version > g0, o._version > o0) == (not to_out, to_out)
    mxq.grad_norm(grads)
    assert to_out or [g._version for g in grads] == [g0 + 1 for g0, _ in before]


def test_a_backward_pass_over_clipped_values_raises():
    x = torch.ones(64, device="cuda", requires_grad=True)
    h = x * 2.0
    loss = (h * h).sum()        # keeps h
    with torch.no_grad():
        mxq.clip_grad_norm([h.detach()], 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_clipped():
    with torch.inference_mode():
        g = torch.ones(100, device="cuda")
        assert mxq.clip_grad_norm([g], 5.0).item() == 10.0
        assert bool((g == 0.5).all())


def test_results_given_by_the_caller_count_a_version():
    T, k, E, N = 20, 2, 4, 32
    plan = plan_of(make_ids(T, k, E, 1), E)
    rows = plan.src.numel()
    y, w, grad = torch.randn((rows, N)).cuda(), torch.rand((T, k)).cuda(), torch.randn((T, N)).cuda()
    out, gy, gw = torch.empty_like(grad), torch.empty_like(y), torch.empty_like(w)
    v = out._version, gy._version, gw._version
    mxq.moe_combine(y, plan, w, out=out)
    mxq.moe_combine_backward(grad, y, plan, w, grad_y=gy, grad_weights=gw)
    assert (out._version, gy._version, gw._version) == tuple(n + 1 for n in v)
    x = torch.randn((rows, 32)).to(torch.bfloat16).cuda()
    l, ls = mxq.quantize_axis(x, "e4m3fn", -1, dense_scale=True)
    d, ds = mxq.quantize_axis(x, "e4m3fn", -2, dense_scale=True)
    wt = torch.randn((32, N)).to(torch.bfloat16).cuda()
    r, rs = (torch.stack([t] * E) for t in mxq.quantize_axis(wt, "e4m3fn", -2, dense_scale=True))
    o1 = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    o2 = torch.empty((E, 32, 32), dtype=torch.bfloat16, device="cuda")
    v = o1._version, o2._version
    mxq.grouped_scaled_matmul(l, ls, r, rs, plan.offsets, out=o1)
    mxq.grouped_scaled_matmul_wgrad(d, ds, d, ds, plan.offsets, out=o2)
    assert (o1._version, o2._version) == tuple(n + 1 for n in v)
