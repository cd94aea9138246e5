"""Plain NumPy definitions of the 8-bit integer form and of the balance loss (test infrastructure only).

quantise and rms_norm decide codes as the header defines them: the fp32 quotient x / s to the nearest whole number, ties
to even. Everything else is fp64.
"""
import numpy as np


def pitch(cols):
    return -(-cols // 16) * 16


def quantise(x):
    """(codes, scales) of fp32 rows."""
    x = np.asarray(x, np.float32)
    s = (np.abs(x).max(1, initial=0) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.where(s[:, None] > 0, x / s[:, None], 0).astype(np.float32)
    return np.clip(np.rint(q), -127, 127).astype(np.int8), s


def stored(codes):
    """codes with zeros up to the pitch"""
    return np.pad(codes, [(0, 0)] * (codes.ndim - 1) + [(0, pitch(codes.shape[-1]) - codes.shape[-1])])


def rms_norm(h, gain, eps):
    """(y, rstd) in fp64, before the rounding to whole numbers"""
    h = np.asarray(h, np.float64)
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * gain, rstd


def rms_norm_grad(dy, h, gain, rstd, dh):
    """(dx, dgain) by the formula"""
    u, v = h * rstd[:, None], dy * gain
    return (0 if dh is None else dh) + rstd[:, None] * (v - u * (u * v).mean(1, keepdims=True)), (dy * u).sum(0)


def matmul(xc, xs, wc, ws, offsets=None, relu=False):
    """Y in fp64; the sums are exact whole numbers"""
    xc, wc = xc.astype(np.int64), wc.astype(np.int64)
    if offsets is None:
        y = (xc @ wc.T).astype(np.float64) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    else:
        y = np.zeros((xc.shape[0], wc.shape[1]))
        for e in range(len(offsets) - 1):
            a, b = offsets[e], offsets[e + 1]
            y[a:b] = matmul(xc[a:b], xs[a:b], wc[e], ws[e])
    return np.maximum(y, 0) if relu else y


def softmax(z):
    m = z.max(1, keepdims=True)
    p = np.where(np.isneginf(m), 0, np.exp(z - np.where(np.isneginf(m), 0, m)))
    s = p.sum(1, keepdims=True)
    return p / np.where(s == 0, 1, s)


def balance(z, ids, mask=None):
    """(loss, counts, p)"""
    experts, top = z.shape[1], ids.shape[1]
    live = np.ones(len(z), bool) if mask is None else mask.astype(bool)
    p = np.zeros(z.shape)
    p[live] = softmax(z[live].astype(np.float64))
    counts = np.zeros(experts + 1, np.int64)
    for t in np.nonzero(live)[0]:
        for e in ids[t]:
            if 0 <= e < experts:
                counts[e] += 1
    counts[-1] = live.sum()
    n = max(1, counts[-1])
    return experts / (top * float(n) ** 2) * (counts[:-1] * p.sum(0)).sum(), counts, p


def balance_grad(dloss, p, counts, top):
    n, c = max(1, counts[-1]), counts[:-1].astype(np.float64)
    return dloss * p.shape[1] / (top * float(n) ** 2) * p * (c - (p * c).sum(1, keepdims=True))
