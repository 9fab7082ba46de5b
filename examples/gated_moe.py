"""A gated mixture-of-experts layer from training to serving, on MX operands.

    python examples/gated_moe.py

Each token goes to `slots` of the experts; an expert is
x -> (silu(x @ Wg) * (x @ Wu)) @ W2 with W1 = [Wg | Wu]. Training runs its products
on FP8 operands; between them the activation is quantized in one pass that keeps its
input in 8 bits, and the backward pass starts from that. Serving quantizes the weights to
e2m1 once: a prompt's tokens go through grouped products, a decode step through two
kernels for the whole layer, captured in a graph.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mx_microscaling_quantization_amd as mxq  # noqa: E402

FMT = "e4m3fn"


def weights_of(w, fmt, dim):
    """Every expert's matrix quantized along dim, with dense scales."""
    return tuple(torch.stack(t) for t in zip(*[mxq.quantize_axis(e, fmt, dim, dense_scale=True) for e in w]))


class GatedMoE:
    """w1 [experts, K, 2F] and w2 [experts, F, K], bfloat16."""

    def __init__(self, w1, w2):
        self.experts = w1.shape[0]
        self.q = {(n, d): weights_of(w, FMT, d) for n, w in (("w1", w1), ("w2", w2)) for d in (-1, -2)}
        self.served = weights_of(w1, "e2m1", -2) + weights_of(w2, "e2m1", -2)

    def forward(self, x, ids, weights):
        plan = mxq.moe_sort(ids, self.experts)
        z = mxq.grouped_scaled_matmul(*mxq.moe_gather_quantize(x, plan, FMT), *self.q["w1", -2], plan.offsets, FMT)
        h, kept = mxq.act_quantize(z, "swiglu", FMT)     # z itself is not kept
        y = mxq.grouped_scaled_matmul(*h, *self.q["w2", -2], plan.offsets, FMT)
        return mxq.moe_combine(y, plan, weights), (x, plan, weights, kept, y)

    def backward(self, grad, saved):
        """Gradients of x, the combine's weights, w1 and w2."""
        x, plan, weights, kept, y = saved
        dy, dweights = mxq.moe_combine_backward(grad, y, plan, weights)
        rows, cols = (mxq.quantize_axis(dy, FMT, d, dense_scale=True) for d in (-1, -2))
        dh = mxq.grouped_scaled_matmul(*rows, *self.q["w2", -1], plan.offsets, FMT)
        dz = mxq.act_quantize_backward(dh, *kept, "swiglu", FMT, FMT)
        dw2 = mxq.grouped_scaled_matmul_wgrad(*dz.h, *cols, plan.offsets, FMT)
        dx = mxq.grouped_scaled_matmul(*dz.rows, *self.q["w1", -1], plan.offsets, FMT)
        dw1 = mxq.grouped_scaled_matmul_wgrad(*mxq.moe_gather_quantize(x, plan, FMT, dim=-2), *dz.cols, plan.offsets,
                                              FMT)
        return mxq.moe_combine(dx, plan), dweights, dw1, dw2

    def prefill(self, x, ids, weights):
        """Many tokens, with the served weights."""
        w1, s1, w2, s2 = self.served
        plan = mxq.moe_sort(ids, self.experts)
        z = mxq.grouped_scaled_matmul_fp4(*mxq.moe_gather_quantize(x, plan, FMT), w1, s1, plan.offsets, FMT)
        h, _ = mxq.act_quantize(z, "swiglu", FMT)
        return mxq.moe_combine(mxq.grouped_scaled_matmul_fp4(*h, w2, s2, plan.offsets, FMT), plan, weights)

    def decode(self, x, ids, weights):
        """A few tokens, with the served weights."""
        return mxq.moe_few_tokens(x, ids, weights, *self.served)


def reference(x, ids, weights, w1, w2):
    """The layer in float32, differentiable."""
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g, u = (x[t] @ w1[e]).chunk(2, 1)
        out = out.index_add(0, t, weights[t, j, None] * ((torch.nn.functional.silu(g) * u) @ w2[e]))
    return out


def problem(tokens, slots, experts, K, F, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    top, ids = torch.topk(rand(tokens, experts), slots, dim=1)
    x, grad = rand(tokens, K).to(torch.bfloat16), rand(tokens, K).to(torch.bfloat16)
    return (x, ids, torch.softmax(top, 1), rand(experts, K, 2 * F, scale=K ** -0.5).to(torch.bfloat16),
            rand(experts, F, K, scale=F ** -0.5).to(torch.bfloat16), grad)


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def train(tokens=1000, slots=2, experts=8, K=512, F=1024):
    """One step's result and gradients: relative distances from the float32 layer's."""
    x, ids, weights, w1, w2, grad = problem(tokens, slots, experts, K, F)
    layer = GatedMoE(w1, w2)
    out, saved = layer.forward(x, ids, weights)
    got = (out, *layer.backward(grad, saved))
    leaves = [t.float().requires_grad_() for t in (x, weights, w1, w2)]
    want = reference(leaves[0], ids, *leaves[1:])
    want.backward(grad.float())
    names = ("out", "dx", "dweights", "dw1", "dw2")
    distance = {n: relative(a, b) for n, a, b in zip(names, got, (want.detach(), *[t.grad for t in leaves]))}
    # a weight's gradient is one dot product, whose terms cancel: its distance is in
    # units of the two vectors' lengths
    plan, y = saved[1], saved[4]
    lengths = grad.float().norm(dim=1, keepdim=True) * y[plan.dest.long()].float().norm(dim=2)
    distance["dweights"] = float((got[2] - leaves[1].grad).norm() / lengths.norm())
    return distance


def served_weights(codes, scale):
    """The values that the served weights hold: [experts, K, C] float32."""
    E, P, _ = codes.shape
    word = codes.view(E, P, -1, 2).int()
    word = word[..., 0] | word[..., 1] << 8
    # (a container's nibbles, from the lowest on, are elements 2, 3, 0, 1)
    n = torch.stack([word >> s & 15 for s in (8, 12, 0, 4)], 2).view(E, 4 * P, -1)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    value = table[(n & 7).long()] * (1 - 2 * (n >> 3))
    return value * torch.exp2(scale.repeat_interleave(32, 1).float() - 127)


def serve(tokens=200, slots=2, experts=8, K=512, F=1024, few=8):
    """A prompt and a decode step, each as far from the float32 layer on the served
    weights' values."""
    x, ids, weights, w1, w2, _ = problem(tokens, slots, experts, K, F)
    layer = GatedMoE(w1, w2)
    values = [served_weights(*layer.served[i:i + 2]) for i in (0, 2)]
    want = reference(x.float(), ids, weights, *values)
    few = min(few, tokens)
    return (relative(layer.prefill(x, ids, weights), want),
            relative(layer.decode(x[:few], ids[:few], weights[:few]), want[:few]))


def decode_graph(tokens=4, slots=4, experts=32, K=512, F=256, steps=4):
    """The decode step captured once and replayed for other tokens, with eager steps in
    between; True if every replay equals the same call made directly."""
    x, ids, weights, w1, w2, _ = problem(tokens, slots, experts, K, F)
    layer = GatedMoE(w1, w2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(x, ids, weights)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(x, ids, weights)
    same = True
    for s in range(steps):
        new = problem(tokens, slots, experts, K, F, seed=1 + s)
        for held, t in zip((x, ids, weights), new):
            held.copy_(t)
        graph.replay()
        same &= torch.equal(out, layer.decode(x, ids, weights))
    return same


if __name__ == "__main__":
    print("training, distance from the float32 layer: " + ", ".join("%s %.3f" % d for d in train().items()))
    print("serving, distance from it on the e2m1 weights: prompt %.4f, decode step %.4f" % serve())
    print("decode graph replays equal direct calls: %s" % decode_graph())
