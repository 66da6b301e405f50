"""Plain 64-bit forms of the operators over vocabulary rows, row by row in numpy on the host: what the GPU
results are compared with.  Written from the definitions in include/domino_head.h."""
import numpy as np

NINF = -np.inf


def order(z):
    """Indices of a row from the largest element on: NaN above every number, ties (and -0, +0) by index."""
    z = np.asarray(z, np.float64)
    key = np.where(np.isnan(z), np.inf, z)
    return np.lexsort((np.arange(len(z)), -key, ~np.isnan(z)))


def lse(y):
    y = np.asarray(y, np.float64)
    if np.isnan(y).any():
        return np.nan
    m = y.max()
    if np.isinf(m):
        return m
    return m + np.log(np.exp(y - m).sum())


def log_softmax(y):
    """Of a row with a finite maximum; differences first, so that rows at a type's lowest value keep them."""
    d = np.asarray(y, np.float64) - np.max(y)
    return d - np.log(np.exp(d).sum())


def top(z, k, tau, n_rows=None):
    B, R, V = z.shape
    ids = np.full((B, R, k), -1, np.int64)
    values = np.full((B, R, k), NINF)
    out = np.full((B, R), NINF)
    for b in range(B):
        for r in range(R if n_rows is None else min(R, max(0, n_rows[b]))):
            ids[b, r] = order(z[b, r])[:k]
            values[b, r] = z[b, r][ids[b, r]]
            out[b, r] = lse(np.asarray(z[b, r], np.float64) / tau)
    return ids, values, out


def beam(z, scores, M, eos=-1, finished=None):
    """Scores (64 bits), parent and token of the M best candidates, and the scores of all in that order."""
    B, W, V = z.shape
    got = []
    for b in range(B):
        cand = []
        for w in range(W):
            s, row = float(scores[b, w]), np.asarray(z[b, w], np.float64)
            if s == NINF:
                c, rank = np.full(V, NINF), np.arange(V)
            elif finished is not None and finished[b, w]:
                c = np.full(V, NINF)
                c[eos] = s
                rank = np.concatenate([[eos], np.delete(np.arange(V), eos)])
            else:
                total = lse(row)
                if not s < np.inf or not total < np.inf:
                    c, rank = np.full(V, np.nan), np.arange(V)
                else:
                    c = np.full(V, NINF) if total == NINF else s + log_softmax(row)
                    rank = order(row)
            cand += [(c[v], w, j, v) for j, v in enumerate(rank[:M])]
        cand.sort(key=lambda x: (not np.isnan(x[0]), -x[0] if not np.isnan(x[0]) else 0.0, x[1], x[2]))
        got.append(cand[:M])
    pick = lambda i: np.array([[c[i] for c in g] for g in got])  # noqa: E731
    return pick(0), pick(1), pick(3)


def distill(z, ids, values, teacher_lse, tau, n_rows=None):
    """Loss [B, R] and dloss/dz [B, R, V]; also the scale of each gradient element's terms (for error bounds)."""
    z = np.asarray(z, np.float64)
    B, R, V = z.shape
    loss, grad, size = np.zeros((B, R)), np.zeros(z.shape), np.zeros(z.shape)
    for b in range(B):
        for r in range(R if n_rows is None else min(R, max(0, n_rows[b]))):
            ok = (ids[b, r] >= 0) & (ids[b, r] < V)
            if not ok.any():
                continue
            i, t = ids[b, r][ok], np.asarray(values[b, r][ok], np.float64) / tau
            L = NINF if teacher_lse is None else float(teacher_lse[b, r])
            noise = (abs(L) + 32) * 2.0 ** -24  # of a mass, by the rounding of L
            told = teacher_lse is not None and not (noise > 2.0 ** -6 and L < np.inf)
            if not told:
                L = lse(t)
            if L == NINF and (t == NINF).all():
                continue
            t = log_softmax(t) if not told and np.isfinite(L) else t - L
            p = np.exp(t)
            y = z[b, r] / tau
            total = lse(y)
            if not total < np.inf or np.isnan(p).any():
                loss[b, r], grad[b, r] = np.nan, np.nan
                continue
            logq = np.full(V, NINF) if total == NINF else log_softmax(y)
            q = np.exp(logq)
            rest = max(0.0, 1.0 - p.sum()) if told else 0.0
            other = np.ones(V, bool)
            other[i] = False
            if told and noise <= 2.0 ** -6 and abs(1.0 - p.sum()) <= noise and q[other].sum() <= noise ** 2:
                # a mass that cannot be told from none, and none of the student's
                rest, t, p = 0.0, t - np.log(p.sum()), p / p.sum()
            with np.errstate(divide="ignore", invalid="ignore"):
                kl = sum(pj * (tj - logq[v]) for pj, tj, v in zip(p, t, i) if pj > 0)
                log_rest = lse(logq[other]) if other.any() else NINF
                if rest > 0:
                    kl += rest * (np.log(rest) - log_rest)
            mass = p.sum() + rest
            g = mass * q
            s = mass * q
            if rest > 0 and log_rest > NINF:
                share = np.exp(log_softmax(y[other]))
                g[other] -= rest * share
                s[other] += rest * share
            np.add.at(g, i, -p)
            np.add.at(s, i, p)
            loss[b, r] = tau * tau * kl
            grad[b, r], size[b, r] = tau * g, tau * s
    return loss, grad, size
