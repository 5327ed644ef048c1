"""Expert routing in plain numpy (fp64): test infrastructure, no code shared
with the CUDA path."""
import numpy as np


def sort(ids, experts):
    """Offsets [experts + 1] and positions of a stable counting sort; -1 where
    the id is no expert."""
    flat = np.asarray(ids).reshape(-1)
    counts = np.zeros(experts + 1, dtype=np.int64)
    for e in flat:
        if 0 <= e < experts:
            counts[e + 1] += 1
    offsets = np.cumsum(counts)
    following = offsets.copy()
    positions = np.full(flat.shape, -1, dtype=np.int64)
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            positions[i] = following[e]
            following[e] += 1
    return offsets.astype(np.int32), positions.reshape(np.shape(ids)).astype(np.int32)


def gather(x, positions, out):
    out = np.array(out)
    for t, row in enumerate(positions):
        for p in row:
            if 0 <= p < len(out):
                out[p] = x[t]
    return out


def combine(ys, positions, weights=None):
    y = np.zeros((len(positions), ys.shape[1]))
    for t, row in enumerate(positions):
        for j, p in enumerate(row):
            if 0 <= p < len(ys):
                y[t] += (1.0 if weights is None else float(weights[t, j])) * ys[p].astype(np.float64)
    return y


def combine_grad(dy, ys, positions, weights, dys):
    dys = np.array(dys, dtype=np.float64)
    dw = np.zeros(np.shape(positions))
    for t, row in enumerate(positions):
        for j, p in enumerate(row):
            if 0 <= p < len(ys):
                g = dy[t].astype(np.float64)
                dys[p] = (1.0 if weights is None else float(weights[t, j])) * g
                dw[t, j] = g @ ys[p].astype(np.float64)
    return dys, dw
