"""Plain double-precision definitions of the steps between an expert block's
products (numpy), written from the formulas alone."""
import numpy as np

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}       # half a step, relative


def sort(idx, n):
    """offsets, perm (the live pairs alone) and place of idx [T, K]."""
    flat = idx.reshape(-1)
    place = np.full(flat.size, -1, np.int64)
    offsets, perm = [0], []
    for e in range(n):
        mine = np.flatnonzero(flat == e)
        place[mine] = offsets[-1] + np.arange(mine.size)
        perm.extend(mine)
        offsets.append(offsets[-1] + mine.size)
    return np.array(offsets), np.array(perm, np.int64), place.reshape(idx.shape)


def combine(rows, place, w, base):
    """(y, sum of magnitudes)."""
    live = place >= 0
    r = np.where(live[..., None], rows[np.where(live, place, 0)], 0.0)
    t = r * (1.0 if w is None else w[..., None].astype(np.float64))
    t = np.where(live[..., None], t, 0.0)
    b = 0.0 if base is None else base
    return t.sum(1) + b, np.abs(t).sum(1) + np.abs(b)


def combine_backward(dy, rows, place, w):
    """(row gradients of each pair [T, K, W], dw, sum of dw's magnitudes)."""
    live = place >= 0
    r = np.where(live[..., None], rows[np.where(live, place, 0)], 0.0)
    t = r * dy[:, None, :]
    return w[..., None].astype(np.float64) * dy[:, None, :], t.sum(-1), np.abs(t).sum(-1)


def situ(g, u):
    with np.errstate(over="ignore"):
        return 4.0 * np.tanh(g / 4.0) / (1.0 + np.exp(-g)) * 25.0 * np.tanh(u / 25.0)


def situ_backward(g, u, dh):
    """(dg, du, what dg's two terms add up to without their signs)."""
    with np.errstate(over="ignore"):
        s, n = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    sech = lambda x: 2.0 / (np.exp(np.minimum(np.abs(x), 350.0)) + np.exp(-np.minimum(np.abs(x), 350.0)))
    t, v = np.tanh(g / 4.0), np.tanh(u / 25.0)
    a, b = s * sech(g / 4.0) ** 2, 4.0 * t * s * n
    return dh * 25.0 * v * (a + b), dh * 4.0 * t * s * sech(u / 25.0) ** 2, np.abs(dh * 25.0 * v) * (np.abs(a) + np.abs(b))


def norm_backward(x, dn, g, eps, dres):
    """(dx, dweight, magnitudes of both)."""
    k = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    n, a = x * k, dn * g
    q = (a * n).mean(1, keepdims=True)
    r = 0.0 if dres is None else dres
    dx = r + k * (a - n * q)
    mag = np.abs(r) + k * (np.abs(a) + np.abs(n) * np.abs(a * n).mean(1, keepdims=True))
    return dx, (dn * n).sum(0), mag, np.abs(dn * n).sum(0)
