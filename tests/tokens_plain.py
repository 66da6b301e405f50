"""Plain 64-bit form of token log-probabilities, entropies and their gradient, row by row in numpy on the host: what the
GPU results are compared with, with bounds of their errors.  Written from the definitions in include/domino_head.h.

Bounds, in halves of a float32 step (H = 2^-24).  An exponential exp(-d) has one step of its own (2 H), and its argument
is rounded twice, the factor and the product: 2 d H.  A thread adds at most 128 of them, vector by vector (22 additions
deep at most), all others in 64 bits.  So a sum of exponentials is known to 26 H and 2 d H of each term; a sum of
exponentials times exponents to 28 H and 4 d H of each term's magnitude.  Where the others than the largest come to 1/8
at least, that one was among them in these additions, which rounded its 1 as well: 22 H.  What follows is in 64 bits, but for the
statistics and the gradient: 12 float32 operations at most on an element of it, and the exponential's own errors again.
(The hardware's exponential gives 0 below 2^-126: such an element of the gradient may be off by all of itself.)
"""
import numpy as np

H = 2.0 ** -24
TINY = 2.0 ** -120


def row(z, token, tau):
    """logprob, entropy, their error bounds, log p and the sums' relative error, of a row of logits."""
    z = np.asarray(z, np.float64)
    V = len(z)
    none = dict(logprob=0.0, entropy=0.0, logprob_err=0.0, entropy_err=0.0, logp=np.full(V, -np.inf), live=False, rel=0.0)
    if not 0 <= token < V:
        return none
    if np.isnan(z).any() or z.max() == np.inf:
        nan = np.nan
        return dict(none, logprob=nan, entropy=nan, logp=np.full(V, nan), live=True)
    if z.max() == -np.inf:
        return dict(none, logprob=-np.inf)
    top = int(np.argmax(z))
    d = (z[top] - z) / tau
    e = np.exp(-d)
    e[top] = 0.0
    with np.errstate(invalid="ignore"):
        ed = np.where(e > 0, e * d, 0.0)
        s_err = (e * 26 + 2 * ed).sum() * H
        t_err = np.where(e > 0, ed * (28 + 4 * d), 0.0).sum() * H
    s, t = e.sum(), ed.sum()
    # (a row of several chunks: each has a largest one of its own, whose weight in the row is among the terms above)
    s_err += 22 * H if s >= 0.124 else 0.0
    logp = -d - np.log1p(s)
    entropy = np.log1p(s) + t / (1 + s)
    logprob_err = s_err / (1 + s)
    entropy_err = logprob_err + (t_err + t * s_err / (1 + s)) / (1 + s)
    return dict(logprob=logp[token], entropy=entropy, live=True, logp=logp, rel=s_err / (1 + s), s=s, top=top,
                logprob_err=logprob_err + (abs(logp[token]) * H if np.isfinite(logp[token]) else 0.0) + TINY,
                entropy_err=entropy_err * 1.01 + entropy * 2 * H + TINY)


def gradient(r, token, tau, g_logprob, g_entropy):
    """The gradient of a row (from row()), and its error bound before it is rounded to its type."""
    V = len(r["logp"])
    if not r["live"]:
        return np.zeros(V), np.zeros(V)
    if np.isnan(r["logprob"]):
        return np.full(V, np.nan), np.zeros(V)
    p = np.exp(r["logp"])
    logp = np.where(p > 0, r["logp"], 0.0)
    d = np.where(p > 0, -logp - np.log1p(r["s"]), 0.0)  # (0 for the largest)
    grad = -p * g_logprob - g_entropy * p * (logp + r["entropy"])
    size = p * (abs(g_logprob) + abs(g_entropy) * (np.abs(logp) + r["entropy"] + np.log1p(r["s"])))
    err = size * (16 * H + 3 * np.abs(d) * H + 2 * r["rel"]) + p * abs(g_entropy) * r["entropy_err"]
    err = np.where(np.exp(-d) < 2.0 ** -125, np.abs(grad), err)
    # the token's: from 1 - p, which the largest has as s / (1 + s)
    one_less = r["s"] / (1 + r["s"]) if r["logp"][token] == r["logp"][r["top"]] else 1 - p[token]
    pt = p[token] * (logp[token] + r["entropy"])
    grad[token] = g_logprob * one_less - g_entropy * pt
    share = r["rel"] * (1 + r["s"]) / r["s"] if r["s"] > 0 else 0.0
    err[token] = abs(g_logprob) * one_less * (6 * H + share) + abs(g_entropy) * (
        abs(pt) * 8 * H + p[token] * (r["logprob_err"] * (1 + abs(logp[token]) + r["entropy"]) + r["entropy_err"]))
    return grad / tau, err / tau * 1.01 + TINY
