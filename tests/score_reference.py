"""Token scores in 64 bits, from their definitions: log probability, entropy and
top alternatives of each row of logits, and the gradient of all three."""
import numpy as np


def parts(row, inv_t):
    """z, p and ln p of one row."""
    z = (row - row.max()) * inv_t
    e = np.where(z == -np.inf, 0.0, np.exp(z))
    s = e.sum()
    return z, e / s, z - np.log(s)


def top(row, k):
    """The k largest elements' indexes, ties to the lowest."""
    return np.argsort(-row, kind="stable")[:k]


def scores(x, y, inv_t, k):
    t = len(y)
    logp, entropy = np.zeros(t), np.zeros(t)
    idx, top_logp = np.full((t, k), -1), np.zeros((t, k))
    for i in range(t):
        if y[i] < 0:
            continue
        _, p, lp = parts(x[i], inv_t)
        logp[i] = lp[y[i]]
        entropy[i] = -(p[p > 0] * lp[p > 0]).sum()
        idx[i] = top(x[i], k)
        top_logp[i] = lp[idx[i]]
    return logp, entropy, idx, top_logp


def gradient(x, y, inv_t, idx, d_logp, d_entropy, d_top):
    grad = np.zeros(x.shape)
    for i in range(len(y)):
        if y[i] < 0:
            continue
        _, p, lp = parts(x[i], inv_t)
        h = -(p[p > 0] * lp[p > 0]).sum()
        lp = np.where(p > 0, lp, 0.0)
        g = -p * (d_logp[i] + d_top[i].sum() + d_entropy[i] * (lp + h))
        g[y[i]] += d_logp[i]
        for j, v in enumerate(idx[i]):
            if 0 <= v < x.shape[1]:
                g[v] += d_top[i, j]
        grad[i] = inv_t * g
    return grad
