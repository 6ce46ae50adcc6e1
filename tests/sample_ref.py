"""Drawing a token from a row of logits in 64 bits, from the definition (include/qlin.h)."""
import numpy as np


def draw(x, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, its share, words left, how near the nearest decision was as a part of the sum, the root of the sum of the
    weights' squares as a part of it)"""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any() or np.isnan(t):
        return -1, 0.0, 0, 1.0, 1.0
    if t <= 0:
        return int(x.argmax()), 1.0, 1, 1.0, 1.0
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp((x - x.max()) / np.float64(t)) if np.isfinite(t) else np.ones_like(x)
    w[x == -np.inf] = 0.0
    order = np.argsort(-x, kind="stable")
    order = order[: int((x > -np.inf).sum())]
    near = 1.0
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1.0:
        run = np.cumsum(w[order])
        need = max(np.float64(top_p), 0.0) * run[-1]
        n = 1 + int((run < need).sum())
        if n > 1 or need > 0:
            near = min(near, np.abs(run - need).min() / run[-1])
        order = order[: min(n, len(order))]
    if min_p > 0:
        m = min(np.float64(min_p), 1.0)
        # (decided by the logits, in 64 bits, not by sums: only a weight within 1e-13 of the bound is near it)
        if m < 1 and (np.abs(w[order] - m) <= 1e-13 * m).any():
            near = 2e-15
        order = order[w[order] >= m]
    ids = np.sort(order)
    run = np.cumsum(w[ids])
    at = np.float64(max(u, 0.0)) * run[-1]
    near = min(near, np.abs(run - at).min() / run[-1] if u < 1 else 1.0)
    n = int((run <= at).sum())
    if n >= len(ids):  # the last word with a weight
        n = int(np.nonzero(w[ids] > 0)[0][-1])
    return int(ids[n]), float(w[ids[n]] / run[-1]), len(ids), float(near), float(np.sqrt((w[ids] ** 2).sum()) / run[-1])
