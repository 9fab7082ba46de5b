"""Products of 4-bit weights, a whole mixture-of-experts layer for a few tokens, and
activations kept in 8 bits, as measured workloads.

Each case is one call a training or serving program makes: the block-scaled product of
activations with e2m1 weights (one matrix, or one per expert), the layer that takes a few
tokens of a decode step through their experts, and a gated activation whose result is
MX-quantized for the next product while its input is kept in 8 bits, with the backward
pass that reads it. With ``own`` false ``run`` computes them with elementary torch
operations; with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

# Exponent of the largest normal value, largest value, mantissa bits, smallest
# normal exponent and bytes of four codes.
FORMATS = {
    "e4m3fn": dict(emax=8, top=448.0, mantissa=3, emin=-6, four=4, torch=torch.float8_e4m3fn),
    "e5m2": dict(emax=15, top=57344.0, mantissa=2, emin=-14, four=4, torch=torch.float8_e5m2),
    "e2m1": dict(emax=2, top=6.0, mantissa=1, emin=0, four=2, torch=None),
}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a dense layer, 4-bit weights, a batch of five
        dict(name="fp4-decode", op="fp4", M=5, K=4096, N=4096, lhs="e4m3fn"),
        # a prefill of odd length through a layer whose sizes fill no tile
        dict(name="fp4-prefill-odd", op="fp4", M=1100, K=4000, N=2052, lhs="e5m2"),
        # both operands in 4 bits, large
        dict(name="fp4-large", op="fp4", M=8192, K=8192, N=8192, lhs="e2m1"),
        # decode: a few rows for each of many experts, bound by the weights
        dict(name="fp4-experts-decode", op="fp4_grouped", T=32, k=8, E=64, K=4096, N=2048, lhs="e4m3fn"),
        # prefill: thousands of rows for each expert, uneven
        dict(name="fp4-experts-prefill", op="fp4_grouped", T=8192, k=4, E=16, K=4096, N=4096, lhs="e4m3fn"),
        # a single token through eight experts of many
        dict(name="layer-one-token", op="layer", T=1, k=8, E=128, K=2048, F=768, N=2048, fmt="e2m1", act="swiglu",
             dtype="bf16", local=1.0),
        # a small batch with 8-bit weights, most experts in use
        dict(name="layer-batch", op="layer", T=16, k=4, E=32, K=4096, F=2048, N=4096, fmt="e4m3fn", act="swiglu",
             dtype="bf16", local=1.0),
        # speculated tokens on a rank that holds half of the experts, odd sizes, no gate
        dict(name="layer-odd", op="layer", T=61, k=6, E=64, K=2016, F=1440, N=2012, fmt="e2m1", act="silu",
             dtype="f16", local=0.5),
        # the activation between the two products of a training step
        dict(name="act-train", op="act", R=16384, F=4096, act="swiglu", dtype="bf16", out="e4m3fn", saved="e4m3fn"),
        # a small layer's, no gate
        dict(name="act-small", op="act", R=40, F=96, act="silu", dtype="f16", out="e5m2", saved="e4m3fn"),
        # its backward pass in the same training step
        dict(name="act-backward-train", op="act_backward", R=16384, F=4096, act="swiglu", dtype="bf16", out="e4m3fn",
             saved="e4m3fn"),
        # the backward pass of a small batch
        dict(name="act-backward-odd", op="act_backward", R=1056, F=1440, act="swiglu", dtype="f16", out="e5m2",
             saved="e5m2"),
    ]


def _spread(rng, low, high):
    """A whole number, spread evenly over the logarithm of low..high."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["fp4", "fp4", "fp4_grouped", "layer", "layer", "act", "act_backward"])
    if op == "fp4":
        K, N = 32 * _spread(rng, 2, 256), 4 * _spread(rng, 8, 2048)
        M = _spread(rng, 1, min(8192, max(1, (1 << 38) // (K * N))))
        return dict(op=op, M=M, K=K, N=N, lhs=rng.choice(["e2m1", "e4m3fn", "e5m2"]))
    k = rng.randint(1, 8)
    E = _spread(rng, max(k, 2), 128)
    if op == "fp4_grouped":
        K, N = 32 * _spread(rng, 2, 128), 4 * _spread(rng, 8, 1024)
        E = min(E, max(k, (1 << 28) // (K * N), 2))
        T = _spread(rng, 1, min(8192, max(1, (1 << 38) // (k * K * N))))
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, lhs=rng.choice(["e2m1", "e4m3fn", "e5m2"]))
    if op == "layer":
        K, F = 32 * _spread(rng, 4, 128), 32 * _spread(rng, 2, 64)
        N = rng.choice([K, K - 4 * rng.randint(0, 7)])
        E = min(E, max(k, (1 << 28) // (K * F), 2))
        return dict(op=op, T=_spread(rng, 1, 64), k=k, E=E, K=K, F=F, N=N, fmt=rng.choice(["e2m1", "e4m3fn", "e5m2"]),
                    act=rng.choice(["swiglu", "silu"]), dtype=rng.choice(["bf16", "f16"]),
                    local=rng.choice([1.0, 0.5]))
    F = 32 * _spread(rng, 1, 256)
    R = (32 if op == "act_backward" else 8) * _spread(rng, 1, max(1, min(1024, (1 << 21) // F)))
    return dict(op=op, R=R, F=F, act=rng.choice(["swiglu", "silu"]), dtype=rng.choice(["bf16", "f16"]),
                out=rng.choice(["e4m3fn", "e5m2"]), saved=rng.choice(["e4m3fn", "e5m2"]))


def _width(case):
    """Columns of the first product's result for each column of the activation's."""
    return 2 if case["act"] == "swiglu" else 1


def _stored(count, fmt):
    """Bytes of this many values with their scales."""
    return count * (FORMATS[fmt]["four"] / 4 + 1 / 32)


def work(case):
    op = case["op"]
    if op == "fp4":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": _stored(M * K, case["lhs"]) + _stored(K * N, "e2m1") + 2 * M * N, "flops": 2 * M * K * N}
    if op in ("act", "act_backward"):
        values = case["R"] * case["F"]
        kept = _stored(values * _width(case), case["saved"])
        if op == "act":
            return {"bytes": 2 * values * _width(case) + kept + _stored(values, case["out"]),
                    "flops": 8 * values * _width(case)}
        return {"bytes": 2 * values + kept + _stored(values * (1 + 2 * _width(case)), case["out"]),
                "flops": 12 * values * _width(case)}
    pairs, E, K = case["T"] * case["k"], case["E"], case["K"]
    if op == "fp4_grouped":
        N = case["N"]
        active = E * (1.0 - (1.0 - 1.0 / E) ** pairs)
        return {"bytes": _stored(pairs * K, case["lhs"]) + _stored(active * K * N, "e2m1") + 2 * pairs * N,
                "flops": 2 * pairs * K * N}
    pairs, E = pairs * case["local"], E * case["local"]
    active = E * (1.0 - (1.0 - 1.0 / E) ** pairs)
    each = case["F"] * (_width(case) * K + case["N"])
    return {"bytes": _stored(active * each, case["fmt"]) + 2 * case["T"] * (K + case["N"]), "flops": 2 * pairs * each}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _experts(case, g):
    """[T, k] distinct expert ids, some experts several times as popular as
    others, with the pairs of experts that live elsewhere marked -1, and weights."""
    T, k, E = case["T"], case["k"], case["E"]
    popular = torch.randn(E, generator=g, device="cuda") * 0.7
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    top, ids = torch.topk(popular - torch.log(-torch.log(noise)), k, dim=1)
    weights = torch.softmax(top, dim=1)
    local = case.get("local", 1.0)
    if local < 1.0:
        ids = torch.where(ids < max(1, int(E * local)), ids, -1)
    return ids, weights


def _activations(shape, g):
    """Normal values with a few columns tens of times as large."""
    scale = torch.exp(torch.randn(shape[-1], generator=g, device="cuda"))
    return torch.randn(shape, generator=g, device="cuda") * scale


def _weight(K, N, fmt, g):
    return _quantize(torch.randn((K, N), generator=g, device="cuda") / math.sqrt(K), fmt, -2)


def _stack(pairs):
    return tuple(torch.stack(t) for t in zip(*pairs))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, state = case["op"], dict(case=case)
    if op == "fp4":
        state["lhs"] = _quantize(_activations((case["M"], case["K"]), g), case["lhs"], -1)
        state["rhs"] = _weight(case["K"], case["N"], "e2m1", g)
    elif op == "fp4_grouped":
        ids, _ = _experts(case, g)
        counts = torch.bincount(ids.reshape(-1), minlength=case["E"])
        ends = torch.cumsum((counts + 31) // 32 * 32, 0)
        state["offsets"] = torch.cat([ends.new_zeros(1), ends]).int()
        pairs = ids.numel()
        rows = (pairs + min(case["E"], pairs) * 31) // 32 * 32
        # the rows that a group's last block leaves empty are zeros, as are those past the last group
        first = state["offsets"][:-1].long()
        place = torch.repeat_interleave(first - (torch.cumsum(counts, 0) - counts), counts)
        x = torch.zeros((rows, case["K"]), device="cuda")
        x[place + torch.arange(pairs, device="cuda")] = _activations((pairs, case["K"]), g)
        state["lhs"] = _quantize(x, case["lhs"], -1)
        state["rhs"] = _stack([_weight(case["K"], case["N"], "e2m1", g) for _ in range(case["E"])])
    elif op == "layer":
        K, F, N, fmt = case["K"], case["F"], case["N"], case["fmt"]
        state["ids"], state["weights"] = _experts(case, g)
        state["x"] = torch.randn((case["T"], K), generator=g, device="cuda").to(DTYPES[case["dtype"]])
        state["w1"] = _stack([_weight(K, F * _width(case), fmt, g) for _ in range(case["E"])])
        state["w2"] = _stack([_weight(F, N, fmt, g) for _ in range(case["E"])])
    else:
        R, F, dtype = case["R"], case["F"], DTYPES[case["dtype"]]
        z = torch.randn((R, F * _width(case)), generator=g, device="cuda") * 1.5
        if op == "act":
            state["z"] = z.to(dtype)
        else:
            state["saved"] = _keep(z, case["saved"])
            state["grad"] = (_activations((R, F), g) * 1e-3).to(dtype)
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _narrow(blocks, dims, fmt):
    """Values on the format's grid and E8M0 bytes of float32 blocks over dims."""
    f = FORMATS[fmt]
    field = (blocks.view(torch.int32) >> 23) & 0xFF
    e8m0 = (field.amax(dims, keepdim=True) - f["emax"]).clamp(min=1)
    scaled = (blocks * ((254 - e8m0) << 23).view(torch.float32)).clamp(-f["top"], f["top"])
    return scaled, e8m0.to(torch.uint8)


def _fp4_codes(scaled):
    """[..., 4] values up to 6 as the two bytes of a container: elements 2 and 3, then 0 and 1."""
    size = scaled.abs()
    step = torch.where(size < 2.0, 0.5, torch.where(size < 4.0, 1.0, 2.0))
    rounded = torch.round(size / step) * step
    index = torch.where(rounded < 2.0, 2.0 * rounded, torch.where(rounded < 4.0, rounded + 2.0, rounded / 2.0 + 4.0))
    code = index.to(torch.uint8) | (torch.signbit(scaled).to(torch.uint8) << 3)
    return torch.stack([code[..., 2] | (code[..., 3] << 4), code[..., 0] | (code[..., 1] << 4)], -1)


def _quantize(x, fmt, dim):
    """MX codes and dense E8M0 bytes of a row-major [R, C] tensor with blocks of 32 along dim:
    [K/4, O containers] and [K/32, O] (K the block axis, O the other)."""
    v = x.float()
    v = (v if dim == -1 else v.t()).contiguous()
    O, K = v.shape
    scaled, e8m0 = _narrow(v.view(O, K // 32, 32), 2, fmt)
    scaled = scaled.view(O, K // 4, 4)
    codes = _fp4_codes(scaled) if fmt == "e2m1" else scaled.to(FORMATS[fmt]["torch"]).view(torch.uint8)
    codes = codes.transpose(0, 1).reshape(K // 4, -1)
    return codes.contiguous(), e8m0.view(O, K // 32).t().contiguous()


def _keep(x, fmt):
    """FP8 codes [R, W] and dense scales [R/8, W/4] with blocks of 8 rows x 4 columns."""
    R, W = x.shape
    scaled, e8m0 = _narrow(x.float().view(R // 8, 8, W // 4, 4), (1, 3), fmt)
    return scaled.to(FORMATS[fmt]["torch"]).view(torch.uint8).view(R, W), e8m0.view(R // 8, W // 4)


def _scale(bytes_):
    return (bytes_.int() << 23).view(torch.float32)


def _decode(codes, scales, fmt):
    """The [K, O] float32 matrix of quantized codes and dense scales."""
    P, O = codes.shape[0], scales.shape[1]
    if fmt == "e2m1":
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        table = torch.cat([table, -table])
        pair = codes.view(P, O, 2)
        values = torch.stack([pair[..., 1] & 15, pair[..., 1] >> 4, pair[..., 0] & 15, pair[..., 0] >> 4], -1)
        values = table[values.int()]
    else:
        values = codes.view(FORMATS[fmt]["torch"]).float().view(P, O, 4)
    return values.transpose(1, 2).reshape(4 * P, O) * _scale(scales).repeat_interleave(32, 0)


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _act(z, act):
    if act == "silu":
        return _silu(z)
    F = z.shape[-1] // 2
    return _silu(z[..., :F]) * z[..., F:]


def _as_values(codes, scales, fmt):
    """The bytes as the numbers they stand for."""
    return codes.view(FORMATS[fmt]["torch"]), scales.view(torch.float8_e8m0fnu)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "fp4":
        return (_decode(*state["lhs"], case["lhs"]).t() @ _decode(*state["rhs"], "e2m1")).to(torch.bfloat16)
    if op == "fp4_grouped":
        left, rhs, offsets = _decode(*state["lhs"], case["lhs"]), state["rhs"], state["offsets"].tolist()
        out = torch.zeros((left.shape[1], case["N"]), dtype=torch.bfloat16, device=left.device)
        for e in range(case["E"]):
            a, b = offsets[e], offsets[e + 1]
            if b > a:
                out[a:b] = (left[:, a:b].t() @ _decode(rhs[0][e], rhs[1][e], "e2m1")).to(torch.bfloat16)
        return out
    if op == "layer":
        x, ids, w1, w2, fmt = state["x"].float(), state["ids"], state["w1"], state["w2"], case["fmt"]
        out = torch.zeros((case["T"], case["N"]), device=x.device)
        for e in torch.unique(ids[ids >= 0]).tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            h = _act(x[t] @ _decode(w1[0][e], w1[1][e], fmt), case["act"])
            out.index_add_(0, t, state["weights"][t, j, None] * (h @ _decode(w2[0][e], w2[1][e], fmt)))
        return out.to(state["x"].dtype)
    out_fmt, act = case["out"], case["act"]
    if op == "act":
        z = state["z"]
        h = _act(z.float(), act).to(z.dtype)
        return _as_values(*_quantize(h, out_fmt, -1), out_fmt) + _as_values(*_keep(z, case["saved"]), case["saved"])
    codes, scales = state["saved"]
    z = codes.view(FORMATS[case["saved"]]["torch"]).float()
    z = z * _scale(scales).repeat_interleave(8, 0).repeat_interleave(4, 1)
    da = state["grad"].float()
    gate = z[:, :case["F"]]
    s = 1.0 / (1.0 + torch.exp(-gate))
    slope = s * (1.0 + gate * (1.0 - s))
    if act == "swiglu":
        dz = torch.cat([da * z[:, case["F"]:] * slope, da * gate * s], 1)
    else:
        dz = da * slope
    dz, h = dz.to(state["grad"].dtype), _act(z, act).to(state["grad"].dtype)
    return (_as_values(*_quantize(dz, out_fmt, -1), out_fmt) + _as_values(*_quantize(dz, out_fmt, -2), out_fmt) +
            _as_values(*_quantize(h, out_fmt, -2), out_fmt))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _run_own(state):
    import mx_microscaling_quantization_amd as mxq

    case = state["case"]
    op = case["op"]
    if op == "fp4":
        return mxq.scaled_matmul_fp4(*state["lhs"], *state["rhs"], case["lhs"], torch.bfloat16, dense_scale=True)
    if op == "fp4_grouped":
        return mxq.grouped_scaled_matmul_fp4(*state["lhs"], *state["rhs"], state["offsets"], case["lhs"],
                                             torch.bfloat16)
    if op == "layer":
        return mxq.moe_few_tokens(state["x"], state["ids"], state["weights"], *state["w1"], *state["w2"], case["fmt"],
                                  case["act"])
    if op == "act":
        out, saved = mxq.act_quantize(state["z"], case["act"], case["out"], case["saved"])
        return _as_values(*out, case["out"]) + _as_values(*saved, case["saved"])
    grads = mxq.act_quantize_backward(state["grad"], *state["saved"], case["act"], case["saved"], case["out"])
    return sum((_as_values(*pair, case["out"]) for pair in grads), ())


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def _power(n):
    """2^n as float64, exactly."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_blocks(v, dims, fmt):
    """Values on the format's grid, and scales, of float64 blocks over dims."""
    f = FORMATS[fmt]
    top = v.abs().amax(dims, keepdim=True)
    _, exponent = torch.frexp(top)                       # top = m * 2^exponent, m in [1/2, 1)
    biased = torch.where(top >= 2.0 ** -126, exponent + 126, 0)
    scale = _power(torch.clamp(biased - f["emax"], min=1) - 127)
    u = v / scale
    _, ue = torch.frexp(u)
    step = _power(torch.clamp(ue - 1, min=f["emin"]) - f["mantissa"])
    return torch.clamp(torch.round(u / step) * step, -f["top"], f["top"]), scale


def _exact_along(v, fmt):
    """The quantized layout of [O, K] float64 rows, blocks of 32 along K."""
    O, K = v.shape
    values, scale = _exact_blocks(v.reshape(O, K // 32, 32), 2, fmt)
    return values.reshape(O, K // 4, 4).transpose(0, 1).reshape(K // 4, 4 * O), scale[..., 0].t()


def _exact_decode(codes, scales, fmt):
    """[K, O] float64 from the formats' bit fields."""
    f = FORMATS[fmt]
    bits = 3 if fmt == "e2m1" else 7
    m, bias = f["mantissa"], 1 - f["emin"]
    byte = np.arange(2 << bits)
    field, frac = (byte & ((1 << bits) - 1)) >> m, byte & ((1 << m) - 1)
    value = np.where(field > 0, (1 + frac / (1 << m)) * 2.0 ** (field - bias), frac / (1 << m) * 2.0 ** (1 - bias))
    table = torch.from_numpy(np.where(byte >> bits, -value, value)).to(codes.device)
    P, O = codes.shape[0], scales.shape[1]
    if fmt == "e2m1":
        # a container read as one number holds elements 2, 3, 0, 1 from its lowest bits on
        word = codes.view(torch.int16).int().reshape(P, O, 1)
        codes = (word >> torch.tensor([8, 12, 0, 4], device=codes.device)) & 15
    # dimensions (p, column, j) -> row 4 p + j
    values = table[codes.reshape(P, O, 4).long()].transpose(1, 2).reshape(P // 8, 32, O)
    return (values * _power(scales.long() - 127)[:, None, :]).reshape(4 * P, O)


def _exact_activation(z, F, act):
    s = torch.sigmoid(z[:, :F])
    return z[:, :F] * s * (z[:, F:] if act == "swiglu" else 1.0)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "fp4":
        left = _exact_decode(*state["lhs"], case["lhs"]).t().contiguous()
        return left @ _exact_decode(*state["rhs"], "e2m1")
    if op == "fp4_grouped":
        left = _exact_decode(*state["lhs"], case["lhs"]).t().contiguous()
        out = torch.zeros((left.shape[0], case["N"]), dtype=torch.float64, device="cuda")
        offsets = state["offsets"].tolist()
        for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
            if b > a:
                out[a:b] = left[a:b] @ _exact_decode(state["rhs"][0][e], state["rhs"][1][e], "e2m1")
        return out
    F, act = case["F"], case["act"]
    if op == "layer":
        out = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            chosen = (state["ids"] == e).double() * state["weights"].double()
            t = torch.nonzero((state["ids"] == e).any(1))[:, 0]
            if t.numel():
                z = state["x"][t].double() @ _exact_decode(state["w1"][0][e], state["w1"][1][e], case["fmt"])
                y = _exact_activation(z, F, act) @ _exact_decode(state["w2"][0][e], state["w2"][1][e], case["fmt"])
                out[t] += chosen[t].sum(1, keepdim=True) * y
        return out
    R, out_fmt, saved_fmt, dtype = case["R"], case["out"], case["saved"], DTYPES[case["dtype"]]
    if op == "act":
        z = state["z"].double()
        W = z.shape[1]
        h = _exact_activation(z, F, act).to(dtype).double()
        kept, kept_scale = _exact_blocks(z.view(R // 8, 8, W // 4, 4), (1, 3), saved_fmt)
        return _exact_along(h, out_fmt) + (kept.reshape(R, W), kept_scale[:, 0, :, 0])
    codes, scales = state["saved"]
    # (the 8 x 4 blocks of row-major codes, as columns of 32 for the decoder)
    W = codes.shape[1]
    blocks = codes.view(R // 8, 8, W // 4, 4).permute(1, 0, 2, 3).reshape(8, -1)
    z = _exact_decode(blocks, scales.reshape(1, -1), saved_fmt)
    z = z.view(8, 4, R // 8, W // 4).permute(2, 0, 3, 1).reshape(R, W)
    da, s = state["grad"].double(), torch.sigmoid(z[:, :F])
    dz = da * (s + z[:, :F] * s * torch.sigmoid(-z[:, :F]))
    if act == "swiglu":
        dz = torch.cat([dz * z[:, F:], da * z[:, :F] * s], 1)
    dz, h = dz.to(dtype).double(), _exact_activation(z, F, act).to(dtype).double()
    return (_exact_along(dz, out_fmt) + _exact_along(dz.t().contiguous(), out_fmt) +
            _exact_along(h.t().contiguous(), out_fmt))
