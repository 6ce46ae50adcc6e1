"""The paged cache of 4 bits a value in numpy, from its definition (include/qlin.h), and attention over it in 64 bits."""
import numpy as np

SCALES = np.array([(8 + (b & 7)) * 2.0 ** ((b >> 3) - 24) for b in range(256)])
PLACE = np.array([4 * (d // 2) + 16 * (d % 2) for d in range(8)])  # of a dim's code in its word


def quantise(x):
    """x fp32 [..., hd]: (codes in -7 .. 7 [..., hd], scale bytes [..., hd / 32])"""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = np.abs(np.where(np.isnan(g), np.float32(0), g)).max(-1)
    need = (top / np.float32(7)).astype(np.float64)
    b = np.minimum(np.searchsorted(SCALES, need), 255)  # the least scale that is at least `need`
    with np.errstate(over="ignore", invalid="ignore"):
        r = np.rint(g / SCALES[b].astype(np.float32)[..., None])
    code = np.where(np.isnan(g), 0, np.clip(r, -7, 7)).astype(np.int64)
    return code.reshape(x.shape), b.astype(np.uint8)


def pack(code):
    """codes [..., hd] as bytes [..., hd / 2]"""
    w = ((code.astype(np.uint64) + 8).reshape(*code.shape[:-1], code.shape[-1] // 8, 8) << PLACE.astype(np.uint64)).sum(-1)
    return np.ascontiguousarray(w.astype("<u4")).view(np.uint8).reshape(*code.shape[:-1], code.shape[-1] // 2)


def values(codes, scales):
    """the values in 64 bits [..., hd] of bytes [..., hd / 2] and scale bytes [..., hd / 32]"""
    w = np.ascontiguousarray(codes).view("<u4").astype(np.int64)
    c = (w[..., None] >> PLACE & 15) - 8
    return c.reshape(*w.shape[:-1], -1) * np.repeat(SCALES[scales], 32, -1)


def rotate(x, cos, sin):
    """x fp32 [..., hd] by cos, sin [hd / 2]; every product and sum rounded to fp32"""
    a, b = np.split(np.asarray(x, np.float32), 2, -1)
    return np.concatenate((a * cos - b * sin, a * sin + b * cos), -1)


def attend(q, keys, vals, p, window, sinks, n_kv, there=None):
    """one lane in 64 bits: q [H][hd]; keys, vals [>= p + 1][n_kv][hd] by position; there: rows whose page is"""
    H, hd = q.shape
    j = np.arange(p + 1)
    seen = (j > p - window) | (j < sinks) if window else np.ones(p + 1, bool)
    if there is not None:
        seen = seen & there[: p + 1]
    out = np.zeros((H, hd))
    if not seen.any():
        return out
    k, v = keys[: p + 1][seen].astype(np.float64), vals[: p + 1][seen].astype(np.float64)
    for h in range(H):
        g = h // (H // n_kv)
        s = k[:, g] @ q[h].astype(np.float64) / np.sqrt(hd)
        w = np.exp(s - s.max())
        out[h] = (w / w.sum()) @ v[:, g]
    return out
