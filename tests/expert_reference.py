"""The mixture-of-experts calls' definitions in 64 bits (numpy): sorting choices by
expert, rows to experts and back, the experts' products."""
import numpy as np


def sort(idx, experts):
    """(starts, source, place) of idx [T, k]; one choice after the other."""
    t, k = idx.shape
    starts, source = [0], []
    place = np.full((t, k), -1, np.int64)
    for e in range(experts):
        for c in np.flatnonzero(idx.ravel() == e):
            place[c // k, c % k] = len(source)
            source.append(c)
        starts.append(len(source))
    return np.array(starts), np.array(source + [-1] * (t * k - len(source)), np.int64), place


def gather(x, place, rows):
    """rows with x[t] in every row of token t; the others as they were."""
    out = rows.copy()
    for t, j in np.argwhere(place >= 0):
        out[place[t, j]] = x[t]
    return out


def combine(y, place, gates):
    out = np.zeros((place.shape[0], y.shape[1]))
    for t, j in np.argwhere(place >= 0):
        out[t] += gates[t, j] * y[place[t, j]]
    return out


def combine_grad(d_out, y, place, gates, d_y):
    d_y, d_gates = d_y.copy(), np.zeros(place.shape)
    for t, j in np.argwhere(place >= 0):
        d_y[place[t, j]] = gates[t, j] * d_out[t]
        d_gates[t, j] = (d_out[t] * y[place[t, j]]).sum()
    return d_y, d_gates


def product(x, w, starts):
    """y of the rows that an expert owns; NaN elsewhere."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(len(starts) - 1):
        y[starts[e]:starts[e + 1]] = x[starts[e]:starts[e + 1]] @ w[e].T
    return y


def product_grad(d_y, x, w, starts):
    d_x, d_w = np.full(x.shape, np.nan), np.zeros(w.shape)
    for e in range(len(starts) - 1):
        r = slice(starts[e], starts[e + 1])
        d_x[r] = d_y[r] @ w[e]
        d_w[e] = d_y[r].T @ x[r]
    return d_x, d_w
