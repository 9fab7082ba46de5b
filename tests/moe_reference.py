"""Plain references of the mixture-of-experts calls (numpy, 64 bits)."""
import numpy as np


def rows_needed(pairs: int, E: int, align: int) -> int:
    return (pairs + min(E, pairs) * (align - 1)) // align * align


def sort(ids: np.ndarray, E: int, align: int):
    """(offsets, src, dest) of [T, k] expert numbers, pair by pair."""
    flat = ids.reshape(-1).astype(np.int64)
    lists = [[] for _ in range(E)]
    for pair, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(pair)
    src = np.full(rows_needed(flat.size, E, align), -1, np.int32)
    dest = np.full(flat.size, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    for e, pairs in enumerate(lists):
        for n, pair in enumerate(pairs):
            src[offsets[e] + n] = pair
            dest[pair] = offsets[e] + n
        offsets[e + 1] = offsets[e] + -(-len(pairs) // align) * align
    return offsets, src, dest.reshape(ids.shape)


def combine(y, dest, weights):
    """(out, sum of magnitudes) in float64."""
    T, k = dest.shape
    out = np.zeros((T, y.shape[1]))
    mags = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            r = dest[t, j]
            if 0 <= r < y.shape[0]:
                term = float(weights[t, j]) * y[r].astype(np.float64)
                out[t] += term
                mags[t] += np.abs(term)
    return out, mags


def combine_backward(grad, y, src, dest, weights):
    """(grad_y, grad_weights, sum of the dot products' magnitudes)."""
    T, k = dest.shape
    grad_y = np.zeros(y.shape)
    for r, pair in enumerate(src):
        if 0 <= pair < T * k:
            grad_y[r] = float(weights.reshape(-1)[pair]) * grad[pair // k].astype(np.float64)
    grad_w = np.zeros((T, k))
    mags = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = dest[t, j]
            if 0 <= r < y.shape[0]:
                prod = grad[t].astype(np.float64) * y[r].astype(np.float64)
                grad_w[t, j] = prod.sum()
                mags[t, j] = np.abs(prod).sum()
    return grad_y, grad_w, mags
