"""Plain 64-bit forms of the layers on the host, written from the definitions in include/domino_head.h: what the GPU
results are compared with."""
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
