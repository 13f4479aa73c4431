"""The training objectives in 64 bits, written from their definitions in
numpy, one token at a time where that is clearer; no code of the library."""
import numpy as np


def log_softmax(x):
    with np.errstate(invalid="ignore"):
        m = x.max(axis=-1, keepdims=True)
        return x - m - np.log(np.exp(x - m).sum(axis=-1, keepdims=True))


def live_tokens(targets, weights, vocab):
    w = np.ones(len(targets)) if weights is None else np.asarray(weights, np.float64)
    return (targets >= 0) & (targets < vocab) & (w != 0), w


def logprobs(x, targets, inv_t=1.0, weights=None):
    live, _ = live_tokens(targets, weights, x.shape[1])
    out = np.zeros(len(targets))
    for t in np.nonzero(live)[0]:
        out[t] = log_softmax(x[t] * inv_t)[targets[t]]
    return out


def rows_gradient(x, targets, slope, inv_t):
    """d loss / d logits from d loss / d logp; rows of slope None are zero."""
    grad = np.zeros_like(x)
    for t, a in enumerate(slope):
        if a is None:
            continue
        one = np.zeros(x.shape[1])
        one[targets[t]] = 1.0
        grad[t] = a * inv_t * (one - np.exp(log_softmax(x[t] * inv_t)))
    return grad


def policy(x, targets, old, adv, ref, weights, lo, hi, beta, inv_t, scale, mean):
    live, w = live_tokens(targets, weights, x.shape[1])
    lp = logprobs(x, targets, inv_t, weights)
    n = float(w[live].sum())
    f = scale / (n if mean and n != 0 else 1.0)
    pol = kl = 0.0
    slope = [None] * len(targets)
    for t in np.nonzero(live)[0]:
        r = np.exp(lp[t] - old[t])
        free, held = r * adv[t], min(max(r, 1 - lo), 1 + hi) * adv[t]
        pol -= w[t] * min(free, held)
        d = 0.0 if free > held else -free
        if beta:
            u = ref[t] - lp[t]
            kl += w[t] * (np.expm1(u) - u)
            d -= beta * np.expm1(u)
        slope[t] = f * w[t] * d
    stats = np.array([f * (pol + beta * kl), f * pol, f * kl, n])
    return stats, lp, rows_gradient(x, targets, slope, inv_t), slope


def preference(x, targets, starts, ref, weights, kind, beta, smoothing, margin, average, inv_t,
               scale):
    pairs = (len(starts) - 1) // 2
    live, w = live_tokens(targets, weights, x.shape[1])
    lp = logprobs(x, targets, inv_t, weights)
    ratio, length = np.zeros(2 * pairs), np.ones(2 * pairs)
    for s in range(2 * pairs):
        part = [t for t in range(starts[s], starts[s + 1]) if live[t]]
        n = sum(w[t] for t in part)
        if average and n != 0:
            length[s] = n
        ratio[s] = sum(w[t] * (lp[t] - (0 if ref is None else ref[t])) for t in part) / length[s]
    total, slope = 0.0, [None] * len(targets)
    for q in range(pairs):
        h = ratio[q] - ratio[pairs + q]
        if kind == "sigmoid":
            z = beta * h - margin
            total += (1 - smoothing) * np.logaddexp(0, -z) + smoothing * np.logaddexp(0, z)
            d = beta * (1 / (1 + np.exp(-z)) - (1 - smoothing))
        else:
            total += (h - 1 / (2 * beta)) ** 2
            d = 2 * (h - 1 / (2 * beta))
        for s, sign in ((q, 1), (pairs + q, -1)):
            for t in range(starts[s], starts[s + 1]):
                if live[t]:
                    slope[t] = sign * scale / pairs * d * w[t] / length[s]
    stats = np.array([scale * total / pairs,
                      beta * np.mean(ratio[:pairs] - ratio[pairs:])])
    return stats, beta * ratio, lp, rows_gradient(x, targets, slope, inv_t), slope


def route(x, k, score, renorm, scale, balance, bias=None, live=None, starts=None, d_gates=None,
          loss_scale=1.0):
    tokens, experts = x.shape
    live = np.ones(tokens, bool) if live is None else np.asarray(live) != 0
    starts = [0, tokens] if starts is None else list(starts)
    if score == "softmax":
        s = np.exp(log_softmax(x))
        z = np.ones(tokens)
    else:
        s = 1 / (1 + np.exp(-x))
        z = s.sum(1) + 1e-20
    key = x if bias is None else s + bias
    idx = np.full((tokens, k), -1, np.int32)
    gates = np.zeros((tokens, k))
    for t in np.nonzero(live)[0]:
        idx[t] = np.argsort(-key[t], kind="stable")[:k]
        picked = s[t, idx[t]]
        gates[t] = scale * picked / (picked.sum() + 1e-20 if renorm else 1.0)
    seqs = [[t for t in range(a, b) if live[t]] for a, b in zip(starts, starts[1:])]
    full = sum(bool(p) for p in seqs)
    counts, loss, pull = np.zeros(experts, np.int64), 0.0, np.zeros_like(x)
    for part in seqs:
        if not part:
            continue
        n = np.bincount(idx[part].ravel(), minlength=experts)
        coef = balance * experts / (k * len(part) ** 2 * full)
        counts += n
        for t in part:
            q = s[t] / z[t]
            loss += coef * float(n @ q)
            b = loss_scale * coef * n
            pull[t] = b if score == "softmax" else (b - b @ q) / z[t]
    grad = np.zeros_like(x)
    for t in np.nonzero(live)[0]:
        if d_gates is not None:
            picked = s[t, idx[t]]
            if renorm:
                down = picked.sum() + 1e-20
                d = scale * (d_gates[t] - d_gates[t] @ picked / down) / down
            else:
                d = scale * d_gates[t]
            pull[t, idx[t]] += d
        if score == "softmax":
            grad[t] = s[t] * (pull[t] - s[t] @ pull[t])
        else:
            grad[t] = s[t] * (1 - s[t]) * pull[t]
    return idx, gates, counts, loss, grad
