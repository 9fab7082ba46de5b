"""The mixture-of-experts operators as measured workloads.

Each case is one call a training or serving program makes: sorting token-expert
pairs by expert, gathering (and MX-quantizing) token rows into that order, the
experts' products on MX operands, bringing the results back to token order with
their weights (and the gradient of that), and clipping many gradients by their
global norm. With ``own`` false ``run`` computes them with elementary torch
operations; with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

# Exponent of the largest normal value, largest value, mantissa bits and
# smallest normal exponent of the FP8 formats.
FORMATS = {
    "e4m3fn": dict(emax=8, top=448.0, mantissa=3, emin=-6, torch=torch.float8_e4m3fn),
    "e5m2": dict(emax=15, top=57344.0, mantissa=2, emin=-14, torch=torch.float8_e5m2),
}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch: 128 pairs, latency only
        dict(name="sort-decode", op="sort", T=16, k=8, E=128, align=32, ids="int64", local=1.0),
        # a long prefill over an expert-parallel rank that owns half the experts
        dict(name="sort-prefill", op="sort", T=65536, k=8, E=256, align=32, ids="int32", local=0.5),
        # a few speculated tokens of a decode step, odd count
        dict(name="gather-quantize-decode", op="gather_quantize", T=61, k=4, E=32, align=32, K=2048, dtype="bf16",
             fmt="e4m3fn", dim=-1),
        # the left operand of the first product of a training step
        dict(name="gather-quantize-train", op="gather_quantize", T=8192, k=8, E=64, align=32, K=4096, dtype="bf16",
             fmt="e4m3fn", dim=-1),
        # the same rows with blocks down the sorted rows, for the weight gradient; odd row count
        dict(name="gather-quantize-wgrad", op="gather_quantize", T=7001, k=6, E=64, align=32, K=4000, dtype="f16",
             fmt="e5m2", dim=-2),
        # results of a prefill brought back to token order
        dict(name="combine-prefill", op="combine", T=16384, k=4, E=32, align=32, N=4096, dtype="bf16"),
        # its gradient in a training step, row length not a multiple of 16 bytes
        dict(name="combine-backward", op="combine_backward", T=6007, k=8, E=64, align=32, N=2052, dtype="bf16"),
        # decode: a few rows for each of many experts, bound by the weights
        dict(name="matmul-decode", op="matmul", T=32, k=8, E=64, align=32, K=4096, N=2048, fmt="e4m3fn"),
        # training: thousands of rows for each expert, uneven
        dict(name="matmul-train", op="matmul", T=8192, k=4, E=16, align=32, K=4096, N=4096, fmt="e4m3fn"),
        # the weight gradients of the same step
        dict(name="matmul-wgrad", op="matmul_wgrad", T=8192, k=4, E=16, align=32, K=2048, N=4096, fmt="e5m2"),
        # a small model's gradients, odd sizes, mixed types
        dict(name="clip-small", op="clip", tensors=48, numel=20011, dtype="mixed", factor=0.25),
        # the expert weights' gradients of one layer
        dict(name="clip-experts", op="clip", tensors=48, numel=4096 * 2048, dtype="bf16", factor=0.1),
    ]


def _spread(rng, low, high):
    """A whole number, spread evenly over the logarithm of low..high."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["sort", "gather_quantize", "combine", "combine_backward", "matmul", "matmul_wgrad", "clip"])
    k = rng.randint(1, 8)
    E = _spread(rng, max(k, 2), 256)
    align = rng.choice([32, 32, 64, 128])
    if op == "sort":
        return dict(op=op, T=_spread(rng, 1, 65536), k=k, E=E, align=align, ids=rng.choice(["int32", "int64"]),
                    local=rng.choice([1.0, 0.5, 0.125]))
    if op == "clip":
        tensors = _spread(rng, 1, 60)
        return dict(op=op, tensors=tensors, numel=_spread(rng, 1, min(1 << 24, (1 << 28) // tensors)),
                    dtype=rng.choice(["f32", "bf16", "f16", "mixed"]), factor=rng.choice([0.1, 0.5, 2.0]))
    fmt = rng.choice(["e4m3fn", "e5m2"])
    if op == "gather_quantize":
        K = 32 * _spread(rng, 1, 256)
        T = _spread(rng, 1, min(16384, max(1, (1 << 27) // (k * K))))
        E = min(E, max(2, T))
        return dict(op=op, T=T, k=min(k, E), E=E, align=align, K=K, dtype=rng.choice(["bf16", "f16"]), fmt=fmt,
                    dim=rng.choice([-1, -2]))
    if op in ("combine", "combine_backward"):
        N = _spread(rng, 1, 8192)
        T = _spread(rng, 1, min(32768, max(1, (1 << 27) // (k * N))))
        E = min(E, max(2, T))
        return dict(op=op, T=T, k=min(k, E), E=E, align=align, N=N, dtype=rng.choice(["bf16", "f16", "f32"]))
    K, N = 32 * _spread(rng, 2, 128), 4 * _spread(rng, 8, 1024)
    E = min(E, max(k, (1 << 28) // (K * N), 2))
    T = _spread(rng, 1, min(8192, max(1, (1 << 38) // (k * K * N))))
    return dict(op=op, T=T, k=k, E=E, align=align, K=K, N=N, fmt=fmt)


def _rows(pairs, E, align):
    """Rows that hold any assignment of the pairs, every group aligned."""
    return (pairs + min(E, pairs) * (align - 1)) // align * align


def work(case):
    op = case["op"]
    if op == "clip":
        total = sum(n for n, _ in _clip_shapes(case))
        size = sum(n * torch.finfo(d).bits // 8 for n, d in _clip_shapes(case))
        return {"bytes": 2 * size, "flops": 3 * total}
    pairs = case["T"] * case["k"]
    if op == "sort":
        ids = 8 if case["ids"] == "int64" else 4
        return {"bytes": pairs * (ids + 4) + 4 * pairs * case["local"] + 4 * case["E"], "flops": 0}
    if op == "gather_quantize":
        return {"bytes": case["T"] * case["K"] * 2 + pairs * case["K"] * 33 / 32 + 4 * pairs, "flops": 0}
    if op in ("combine", "combine_backward"):
        size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        row = case["N"] * size
        if op == "combine":
            return {"bytes": (pairs + case["T"]) * row + 8 * pairs, "flops": 2 * pairs * case["N"]}
        return {"bytes": (2 * pairs + case["T"]) * row + 12 * pairs, "flops": 3 * pairs * case["N"]}
    K, N, E = case["K"], case["N"], case["E"]
    active = E * (1.0 - (1.0 - 1.0 / E) ** pairs)
    if op == "matmul":
        return {"bytes": pairs * K * 33 / 32 + active * K * N * 33 / 32 + 2 * pairs * N, "flops": 2 * pairs * K * N}
    return {"bytes": pairs * (K + N) * 33 / 32 + 2 * E * K * N, "flops": 2 * pairs * K * N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _experts(case, g):
    """[T, k] distinct expert ids, some experts several times as popular as
    others, with the pairs of experts that live elsewhere marked -1."""
    T, k, E = case["T"], case["k"], case["E"]
    popular = torch.randn(E, generator=g, device="cuda") * 0.7
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    scores = popular - torch.log(-torch.log(noise))
    top, ids = torch.topk(scores, k, dim=1)
    weights = torch.softmax(top, dim=1)
    local = case.get("local", 1.0)
    if local < 1.0:
        ids = torch.where(ids < max(1, int(E * local)), ids, -1)
    return ids, weights


def _sort(ids, E, align):
    """Pairs in expert order: offsets [E + 1], src [rows], dest [T, k]."""
    T, k = ids.shape
    pairs = T * k
    rows = _rows(pairs, E, align)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    counts.index_add_(0, key, torch.ones_like(key))
    padded = (counts[:E] + align - 1) // align * align
    zero = torch.zeros(1, dtype=torch.int64, device=ids.device)
    offsets = torch.cat([zero, torch.cumsum(padded, 0)])
    starts = torch.cat([zero, torch.cumsum(counts, 0)])[:-1]
    sorted_key = key[order]
    position = offsets[sorted_key.clamp(max=E)] + torch.arange(pairs, device=ids.device) - starts[sorted_key]
    routed = sorted_key < E
    src = torch.full((rows + 1,), -1, dtype=torch.int32, device=ids.device)
    src[torch.where(routed, position, rows)] = order.int()
    dest = torch.empty(pairs, dtype=torch.int32, device=ids.device)
    dest[order] = torch.where(routed, position, -1).int()
    return offsets.int(), src[:rows].contiguous(), dest.view(T, k)


def _clip_shapes(case):
    kinds = ["f32", "bf16", "f16"] if case["dtype"] == "mixed" else [case["dtype"]]
    n = case["numel"]
    # odd sizes about the nominal one, where the nominal one is odd
    step = 0 if n % 2 == 0 else max(1, n // 53)
    return [(max(1, n - step * (i % 7)), DTYPES[kinds[i % len(kinds)]]) for i in range(case["tensors"])]


def _activations(shape, dtype, g):
    """Normal values with a few columns tens of times as large."""
    scale = torch.exp(torch.randn(shape[-1], generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "clip":
        grads = [(torch.randn(n, generator=g, device="cuda") * 0.02).to(d) for n, d in _clip_shapes(case)]
        elements = sum(n for n, _ in _clip_shapes(case))
        return dict(case=case, grads=grads, out=[torch.empty_like(t) for t in grads],
                    max_norm=case["factor"] * 0.02 * math.sqrt(elements))
    ids, weights = _experts(case, g)
    if op == "sort":
        return dict(case=case, ids=ids.to(getattr(torch, case["ids"])))
    offsets, src, dest = _sort(ids, case["E"], case["align"])
    state = dict(case=case, offsets=offsets, src=src, dest=dest)
    rows = src.numel()
    if op == "gather_quantize":
        state["x"] = _activations((case["T"], case["K"]), DTYPES[case["dtype"]], g)
    elif op in ("combine", "combine_backward"):
        dtype = DTYPES[case["dtype"]]
        y = torch.randn((rows, case["N"]), generator=g, device="cuda")
        state["y"] = torch.where(src[:, None] >= 0, y, 0.0).to(dtype)
        state["weights"] = weights.contiguous()
        if op == "combine_backward":
            state["grad"] = torch.randn((case["T"], case["N"]), generator=g, device="cuda").to(dtype)
    else:
        K, N, E, fmt = case["K"], case["N"], case["E"], case["fmt"]
        keep = src[:, None] >= 0
        x = torch.where(keep, torch.randn((rows, K), generator=g, device="cuda"), 0.0)
        if op == "matmul":
            state["lhs"] = _quantize(x, fmt, -1)
            state["rhs"] = tuple(
                torch.stack(t) for t in zip(*[
                    _quantize(torch.randn((K, N), generator=g, device="cuda") / math.sqrt(K), fmt, -2)
                    for _ in range(E)]))
        else:
            y = torch.where(keep, torch.randn((rows, N), generator=g, device="cuda"), 0.0)
            state["lhs"] = _quantize(x, fmt, -2)
            state["rhs"] = _quantize(y, fmt, -2)
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _quantize(x, fmt, dim):
    """MX codes and E8M0 bytes of a row-major [R, C] tensor with blocks of 32
    along dim, as the [K/4, 4 O] codes and dense [K/32, O] scales of the
    partition-major view (K the block axis, O the other)."""
    f = FORMATS[fmt]
    v = x.float()
    v = (v if dim == -1 else v.t()).contiguous()
    O, K = v.shape
    blocks = v.view(O, K // 32, 32)
    field = (blocks.view(torch.int32) >> 23) & 0xFF
    e8m0 = (field.amax(-1) - f["emax"]).clamp(min=1)
    scaled = blocks * ((254 - e8m0) << 23).view(torch.float32)[..., None]
    scaled = torch.where(torch.isnan(scaled), torch.copysign(torch.zeros_like(scaled), scaled), scaled)
    codes = scaled.clamp(-f["top"], f["top"]).to(f["torch"]).view(torch.uint8)
    codes = codes.view(O, K // 4, 4).permute(1, 0, 2).reshape(K // 4, 4 * O)
    return codes.contiguous(), e8m0.to(torch.uint8).t().contiguous()


def _decode(codes, scales, fmt):
    """The [K, O] float32 matrix of partition-major codes and dense scales."""
    P, O = codes.shape[0], scales.shape[1]
    values = codes.view(FORMATS[fmt]["torch"]).float().view(P, O, 4).permute(0, 2, 1).reshape(4 * P, O)
    return values * (scales.int() << 23).view(torch.float32).repeat_interleave(32, 0)


def _as_values(codes, scales, fmt):
    """The bytes as the numbers they stand for."""
    return codes.view(FORMATS[fmt]["torch"]), scales.view(torch.float8_e8m0fnu)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "sort":
        return _sort(state["ids"], case["E"], case["align"])
    if op == "clip":
        total = sum(t.double().square().sum() for t in state["grads"])
        norm = torch.sqrt(total)
        factor = torch.where(norm > state["max_norm"], state["max_norm"] / norm, 1.0).float()
        return norm.float(), [(t.float() * factor).to(t.dtype) for t in state["grads"]]
    src, dest, k = state["src"], state["dest"], case["k"]
    token = torch.div(src.clamp(min=0), k, rounding_mode="floor").long()
    if op == "gather_quantize":
        rows = torch.where(src[:, None] >= 0, state["x"][token].float(), 0.0)
        return _as_values(*_quantize(rows, case["fmt"], case["dim"]), case["fmt"])
    if op in ("combine", "combine_backward"):
        y, weights = state["y"], state["weights"]
        routed = dest >= 0
        picked = torch.where(routed[..., None], y[dest.clamp(min=0).long()].float(), 0.0)
        if op == "combine":
            return (picked * weights[..., None]).sum(1).to(y.dtype)
        grad = state["grad"].float()
        grad_weights = (picked * grad[:, None, :]).sum(-1)
        row_weight = torch.where(src >= 0, weights.reshape(-1)[src.clamp(min=0).long()], 0.0)
        return (grad[token] * row_weight[:, None]).to(y.dtype), grad_weights
    offsets = state["offsets"].tolist()
    lhs, rhs = state["lhs"], state["rhs"]
    E, N, fmt = case["E"], case["N"], case["fmt"]
    if op == "matmul":
        left = _decode(*lhs, fmt)
        out = torch.zeros((left.shape[1], N), dtype=torch.bfloat16, device=left.device)
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            if b > a:
                out[a:b] = (left[:, a:b].t() @ _decode(rhs[0][e], rhs[1][e], fmt)).to(torch.bfloat16)
        return out
    left, right = _decode(*lhs, fmt), _decode(*rhs, fmt)
    out = torch.zeros((E, case["K"], N), dtype=torch.bfloat16, device=left.device)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            out[e] = (left[a:b].t() @ right[a:b]).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _run_own(state):
    import mx_microscaling_quantization_amd as mxq

    case = state["case"]
    op = case["op"]
    if op == "sort":
        plan = mxq.moe_sort(state["ids"], case["E"], align=case["align"])
        return plan.offsets, plan.src, plan.dest
    if op == "clip":
        norm = mxq.clip_grad_norm(state["grads"], state["max_norm"], out=state["out"])
        return norm, state["out"]
    plan = mxq.MoEPlan(state["offsets"], state["src"], state["dest"])
    if op == "gather_quantize":
        data, scale = mxq.moe_gather_quantize(state["x"], plan, case["fmt"], dim=case["dim"])
        return _as_values(data, scale, case["fmt"])
    if op == "combine":
        return mxq.moe_combine(state["y"], plan, state["weights"])
    if op == "combine_backward":
        return mxq.moe_combine_backward(state["grad"], state["y"], plan, state["weights"])
    call = mxq.grouped_scaled_matmul if op == "matmul" else mxq.grouped_scaled_matmul_wgrad
    return call(*state["lhs"], *state["rhs"], plan.offsets, case["fmt"], torch.bfloat16)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def _power(n):
    """2^n as float64, exactly."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_quantize(v, fmt):
    """Values on the FP8 grid, and scales, of [O, K] float64 rows."""
    f = FORMATS[fmt]
    O, K = v.shape
    top = v.abs().view(O, K // 32, 32).amax(-1)
    _, exponent = torch.frexp(top)                       # top = m * 2^exponent, m in [1/2, 1)
    biased = torch.where(top >= 2.0 ** -126, exponent + 126, 0)
    e8m0 = torch.clamp(biased - f["emax"], min=1)
    scale = _power(e8m0 - 127)
    u = v / scale.repeat_interleave(32, 1)
    _, ue = torch.frexp(u)
    step = _power(torch.clamp(ue - 1, min=f["emin"]) - f["mantissa"])
    return torch.clamp(torch.round(u / step) * step, -f["top"], f["top"]), scale


def _exact_decode(codes, scales, fmt):
    """[K, O] float64 from the formats' bit fields."""
    f = FORMATS[fmt]
    m, bias = f["mantissa"], 1 - f["emin"]
    byte = np.arange(256)
    field, frac = (byte & 0x7F) >> m, byte & ((1 << m) - 1)
    value = np.where(field > 0, (1 + frac / (1 << m)) * 2.0 ** (field - bias), frac / (1 << m) * 2.0 ** (1 - bias))
    table = torch.from_numpy(np.where(byte & 0x80, -value, value)).to(codes.device)
    P, O = codes.shape[0], scales.shape[1]
    # dimensions (p, column, j) -> row 4 p + j
    values = table[codes.long()].reshape(P, O, 4).transpose(1, 2).reshape(4 * P, O)
    return values.view(P // 8, 32, O).mul(_power(scales.long() - 127)[:, None, :]).view(4 * P, O)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        ids = state["ids"].cpu().numpy().reshape(-1).astype(np.int64)
        E, align = case["E"], case["align"]
        src = np.full(_rows(ids.size, E, align), -1, np.int32)
        dest = np.full(ids.size, -1, np.int32)
        offsets = np.zeros(E + 1, np.int32)
        for e in range(E):
            pairs = np.nonzero(ids == e)[0]
            at = offsets[e] + np.arange(pairs.size)
            src[at], dest[pairs] = pairs, at
            offsets[e + 1] = offsets[e] + -(-pairs.size // align) * align
        return offsets, src, dest.reshape(case["T"], case["k"])
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for t in state["grads"]:
            total += torch.dot(t.double(), t.double())
        norm = total.sqrt()
        factor = min(1.0, state["max_norm"] / norm.item())
        return norm, [t.double() * factor for t in state["grads"]]
    src, dest, k = state["src"].long(), state["dest"].long(), case["k"]
    held = torch.nonzero(src >= 0)[:, 0]
    if op == "gather_quantize":
        rows = torch.zeros((src.numel(), case["K"]), dtype=torch.float64, device="cuda")
        rows[held] = state["x"][src[held] // k].double()
        values, scale = _exact_quantize(rows if case["dim"] == -1 else rows.t().contiguous(), case["fmt"])
        O, K = values.shape
        return values.reshape(O, K // 4, 4).transpose(0, 1).reshape(K // 4, 4 * O), scale.t()
    if op in ("combine", "combine_backward"):
        y, weights = state["y"], state["weights"].double()
        if op == "combine":
            out = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
            for j in range(k):
                t = torch.nonzero(dest[:, j] >= 0)[:, 0]
                out[t] += weights[t, j, None] * y[dest[t, j]].double()
            return out
        grad = state["grad"].double()
        grad_y = torch.zeros((src.numel(), case["N"]), dtype=torch.float64, device="cuda")
        grad_weights = torch.zeros((case["T"], k), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(dest[:, j] >= 0)[:, 0]
            grad_y[dest[t, j]] = weights[t, j, None] * grad[t]
            grad_weights[t, j] = (grad[t] * y[dest[t, j]].double()).sum(-1)
        return grad_y, grad_weights
    offsets = state["offsets"].tolist()
    lhs, rhs, E, N, fmt = state["lhs"], state["rhs"], case["E"], case["N"], case["fmt"]
    left = _exact_decode(*lhs, fmt)
    if op == "matmul":
        out = torch.zeros((left.shape[1], N), dtype=torch.float64, device="cuda")
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            if b > a:
                out[a:b] = left[:, a:b].t().contiguous() @ _exact_decode(rhs[0][e], rhs[1][e], fmt)
        return out
    right = _exact_decode(*rhs, fmt)
    return torch.stack([left[a:b].t().contiguous() @ right[a:b] for a, b in zip(offsets, offsets[1:])])
