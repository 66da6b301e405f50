"""Plain 64-bit forms of the layers on the host, written from the definitions in include/domino_head.h: what the GPU
results are compared with."""
import math

import numpy as np


def embed(table, ids, scale):
    V, d = table.shape
    flat = ids.reshape(-1)
    out = np.zeros((flat.size, d))
    ok = (flat >= 0) & (flat < V)
    out[ok] = scale * np.asarray(table, np.float64)[flat[ok]]
    return out.reshape(ids.shape + (d,))


def embed_backward(grad, ids, V, scale):
    """The sums [V, d], the sums of the terms' magnitudes, and the number of terms of each row."""
    g, flat = np.asarray(grad, np.float64).reshape(-1, grad.shape[-1]), ids.reshape(-1)
    total, size, count = np.zeros((V, g.shape[1])), np.zeros((V, g.shape[1])), np.zeros(V, np.int64)
    for i, v in enumerate(flat):
        if 0 <= v < V:
            total[v] += scale * g[i]
            size[v] += abs(scale) * np.abs(g[i])
            count[v] += 1
    return total, size, count


def _erfc(z):
    return np.vectorize(math.erfc, otypes=[np.float64])(z) if z.size else z


def act(a, name):
    with np.errstate(over="ignore"):
        if name == "silu":
            return a / (1 + np.exp(-a))
        if name == "gelu":
            return 0.5 * a * _erfc(-a / math.sqrt(2))
    return np.maximum(a, 0) if name == "relu" else a


def slope(a, name):
    with np.errstate(over="ignore"):
        if name == "silu":
            s = 1 / (1 + np.exp(-a))
            return s * (1 + a / (1 + np.exp(a)))
        if name == "gelu":
            return 0.5 * _erfc(-a / math.sqrt(2)) + a * np.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    return (a > 0) * 1.0 if name == "relu" else np.ones_like(a)


def product(a, b):
    """a b^T, and the same of magnitudes."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return a @ b.T, np.abs(a) @ np.abs(b).T
