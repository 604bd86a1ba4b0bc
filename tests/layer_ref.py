"""Plain forms in 64 bits of the operators between a layer's products (include/mxnum_layer.h), in numpy, and the bounds on what
FP32 arithmetic and one rounding to BF16 may add to them.

EPS32 and HALF16 are half a step of FP32 and BF16: a rounding is off by at most that share of the value."""
import numpy as np

EPS32, HALF16, TINY16 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -133


def bf16(a):
    """The nearest BF16 value (ties to even) of FP32-representable numbers, as float64."""
    bits = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    up = ((bits + 0x7FFF + ((bits >> 16) & 1)) >> 16).astype(np.uint32)
    out = (up << 16).view(np.float32)
    return np.where(np.isnan(a), np.nan, out).astype(np.float64)


def norm(x, w, eps, residual=None):
    """(h, n, y before its rounding)."""
    h = x if residual is None else bf16((x + residual).astype(np.float32))
    with np.errstate(invalid="ignore", divide="ignore"):
        r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
        return h, h * r, h * r * w


def norm_backward(dy, h, w, eps, dsum=None):
    """(dx, dweight, bound of dx, bound of dweight per added term)."""
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, dn = h * r, dy * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdims=True))
    # a row's sum has a chain of 8 and a tree of 11 levels; r takes half of the sum's 19 roundings and has 4 of its own (14), n one
    # more; mean(dn n) has 1 + 19 in its sum, 3 in the mean and r's 14; n times it 52, less dn, times r 15 more: below 70
    near = 70 * EPS32 * r * (np.abs(dn) + np.abs(n) * np.abs(dn * n).mean(-1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
        near = near + EPS32 * np.abs(dx)
    return dx, (dy * n).sum(0), HALF16 * np.abs(dx) + 1.01 * near + TINY16, np.abs(dy * n).sum(0)


def route(z, k, normalize):
    """(ids, weights): -1 and zero where only -inf is left."""
    t = z.shape[0]
    key = np.where(np.isnan(z), np.inf, z)
    first = np.where(np.isnan(z), 0, 1)
    order = np.lexsort((np.broadcast_to(np.arange(z.shape[1]), z.shape), first, -key), axis=-1)[:, :k]
    picked = np.take_along_axis(z, order, 1)
    out = np.isneginf(picked)
    with np.errstate(invalid="ignore"):
        top = picked[:, :1]
        e = np.where(out, 0.0, np.exp(picked - top))
        every = np.where(np.isneginf(z), 0.0, np.exp(z - top))
        total = (e if normalize else every).sum(-1, keepdims=True)
        w = np.where(out, 0.0, e / np.where(total == 0, 1.0, total))
    return np.where(out, -1, order).astype(np.int32), w


def route_backward(z, ids, dw, normalize):
    """(dlogits, the sum of the magnitudes that it is made of)."""
    t, experts = z.shape
    have = (ids >= 0) & (ids < experts)
    at = np.where(have, ids, 0)
    picked = np.where(have, np.take_along_axis(z, at, 1), -np.inf)
    dw = np.where(have, dw, 0.0)
    top = (picked if normalize else z).max(-1, keepdims=True)
    top = np.where(np.isneginf(top), 0.0, top)
    e, every = np.exp(picked - top), np.exp(z - top)
    total = (e if normalize else every).sum(-1, keepdims=True)
    total = np.where(total == 0, 1.0, total)
    w, p = e / total, every / total
    inner, size = (w * dw).sum(-1, keepdims=True), (w * np.abs(dw)).sum(-1, keepdims=True)
    dz, mag = (np.zeros_like(z), np.zeros_like(z)) if normalize else (-p * inner, p * size)
    for j in range(ids.shape[1]):
        part = w[:, j] * (dw[:, j] - (inner[:, 0] if normalize else 0.0))
        much = w[:, j] * (np.abs(dw[:, j]) + (size[:, 0] if normalize else 0.0))
        np.add.at(dz, (np.arange(t), at[:, j]), np.where(have[:, j], part, 0.0))
        np.add.at(mag, (np.arange(t), at[:, j]), np.where(have[:, j], much, 0.0))
    return dz, mag


def sort(ids, experts):
    """(group_offsets, rows, source)."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(experts + 1))
    rows, source = np.full(flat.size, -1), np.full(flat.size, -1)
    used = offsets[-1]
    rows[order[:used]] = np.arange(used)
    source[:used] = order[:used]
    return offsets.astype(np.int64), rows.reshape(ids.shape).astype(np.int32), source.astype(np.int32)


def combine(z, rows, w=None, residual=None):
    """(y before its rounding, the sum of the magnitudes)."""
    have = (rows >= 0) & (rows < z.shape[0])
    w = np.ones(rows.shape) if w is None else w
    y = np.zeros((rows.shape[0], z.shape[1])) if residual is None else residual.copy()
    mag = np.abs(y)
    for j in range(rows.shape[1]):
        on = have[:, j]
        part = w[on, j, None] * z[rows[on, j]]
        y[on] += part
        mag[on] += np.abs(part)
    return y, mag


def combine_backward(dy, z, rows, w, dz):
    """(dz with the rows that none names as given, dweights, the sum of dweights' magnitudes)."""
    have = (rows >= 0) & (rows < z.shape[0])
    dz, dw, mag = dz.copy(), np.zeros(rows.shape), np.zeros(rows.shape)
    for j in range(rows.shape[1]):
        on = have[:, j]
        dz[rows[on, j]] = w[on, j, None] * dy[on]
        dw[on, j] = (dy[on] * z[rows[on, j]]).sum(-1)
        mag[on, j] = np.abs(dy[on] * z[rows[on, j]]).sum(-1)
    return dz, dw, mag
