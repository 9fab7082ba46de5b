"""One training step of a mixture-of-experts layer whose products run on MX operands.

    python examples/moe_step.py

Each token goes to `slots` of the experts; an expert is x -> silu(x @ W1) @ W2.
Every product -- forward, the gradient of its input, the gradient of its
weights -- takes FP8 operands with E8M0 block scales. The result and the
gradients are compared with a float32 layer's (autograd), and the forward pass
is captured in a graph and replayed for other tokens, as a decode loop would.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mx_microscaling_quantization_amd as mxq  # noqa: E402

FMT = "e4m3fn"


def quantize(x, dim):
    return mxq.quantize_axis(x, FMT, dim, dense_scale=True)


class MoELayer:
    """w1 [experts, K, F] and w2 [experts, F, K], bfloat16; quantized once per
    update, along the contraction of the forward products (dim -2) and of their
    input gradients (dim -1)."""

    def __init__(self, w1, w2):
        self.experts = w1.shape[0]
        self.w1, self.w2 = w1, w2
        self.q = {(n, d): tuple(torch.stack(t) for t in zip(*[quantize(e, d) for e in w]))
                  for n, w in (("w1", w1), ("w2", w2)) for d in (-1, -2)}

    def forward(self, x, ids, weights):
        plan = mxq.moe_sort(ids, self.experts)
        z = mxq.grouped_scaled_matmul(*mxq.moe_gather_quantize(x, plan, FMT), *self.q["w1", -2], plan.offsets, FMT)
        a = torch.nn.functional.silu(z)
        y = mxq.grouped_scaled_matmul(*quantize(a, -1), *self.q["w2", -2], plan.offsets, FMT)
        return mxq.moe_combine(y, plan, weights), (x, plan, weights, z, a, y)

    def backward(self, grad, saved):
        """Gradients of x, the combine's weights, w1 and w2."""
        x, plan, weights, z, a, y = saved
        dy, dweights = mxq.moe_combine_backward(grad, y, plan, weights)
        da = mxq.grouped_scaled_matmul(*quantize(dy, -1), *self.q["w2", -1], plan.offsets, FMT)
        dw2 = mxq.grouped_scaled_matmul_wgrad(*quantize(a, -2), *quantize(dy, -2), plan.offsets, FMT)
        s = torch.sigmoid(z.float())
        dz = (da.float() * s * (1 + z.float() * (1 - s))).to(torch.bfloat16)
        dx = mxq.grouped_scaled_matmul(*quantize(dz, -1), *self.q["w1", -1], plan.offsets, FMT)
        dw1 = mxq.grouped_scaled_matmul_wgrad(*mxq.moe_gather_quantize(x, plan, FMT, dim=-2), *quantize(dz, -2),
                                              plan.offsets, FMT)
        return mxq.moe_combine(dx, plan), dweights, dw1, dw2


def reference(x, ids, weights, w1, w2, grad):
    """The same layer in float32 with autograd: (out, dx, dweights, dw1, dw2)."""
    leaves = [t.float().requires_grad_() for t in (x, weights, w1, w2)]
    x, weights, w1, w2 = leaves
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y = torch.nn.functional.silu(x[t] @ w1[e]) @ w2[e]
        out = out.index_add(0, t, weights[t, j, None] * y)
    out.backward(grad.float())
    return (out.detach(), *[t.grad for t in leaves])


def problem(tokens, slots, experts, K, F, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    top, ids = torch.topk(rand(tokens, experts), slots, dim=1)
    x, grad = rand(tokens, K).to(torch.bfloat16), rand(tokens, K).to(torch.bfloat16)
    return (x, ids, torch.softmax(top, 1), rand(experts, K, F, scale=K ** -0.5).to(torch.bfloat16),
            rand(experts, F, K, scale=F ** -0.5).to(torch.bfloat16), grad)


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def step(tokens=1000, slots=2, experts=8, K=512, F=1024, max_norm=1.0):
    """One step; relative distances from the float32 layer, the gradients'
    norm before clipping and after it."""
    x, ids, weights, w1, w2, grad = problem(tokens, slots, experts, K, F)
    layer = MoELayer(w1, w2)
    out, saved = layer.forward(x, ids, weights)
    got = (out, *layer.backward(grad, saved))
    names = ("out", "dx", "dweights", "dw1", "dw2")
    want = reference(x, ids, weights, w1, w2, grad)
    distance = {n: relative(a, b) for n, a, b in zip(names, got, want)}
    # a weight's gradient is one dot product, whose terms cancel: its distance
    # is in units of the two vectors' lengths
    plan, y = saved[1], saved[5]
    lengths = grad.float().norm(dim=1, keepdim=True) * y[plan.dest.long()].float().norm(dim=2)
    distance["dweights"] = float((got[2] - want[2]).norm() / lengths.norm())
    grads = [g for w in got[3:] for g in w.unbind()]
    norm = mxq.clip_grad_norm(grads, max_norm)
    return distance, float(norm), float(mxq.grad_norm(grads))


def decode_graph(tokens=16, slots=4, experts=32, K=512, F=256, steps=3):
    """The forward pass captured once and replayed for other tokens; True if
    every replay equals the same call made directly."""
    x, ids, weights, w1, w2, _ = problem(tokens, slots, experts, K, F)
    layer = MoELayer(w1, w2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x, ids, weights)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = layer.forward(x, ids, weights)
    same = True
    for s in range(steps):
        new = problem(tokens, slots, experts, K, F, seed=1 + s)
        for held, t in zip((x, ids, weights), new):
            held.copy_(t)
        graph.replay()
        same &= torch.equal(out, layer.forward(x, ids, weights)[0])
    return same


if __name__ == "__main__":
    distance, before, after = step()
    print("distance from the float32 layer: " + ", ".join("%s %.3f" % d for d in distance.items()))
    print("norm of the expert weights' gradients: %.3f, clipped to %.3f" % (before, after))
    print("decode graph replays equal direct calls: %s" % decode_graph())
