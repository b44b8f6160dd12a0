"""Microscaled 4-bit codes, RMS norm and the gated feed-forward block on the CPU, in
64 bits and from the definitions: a table of the e2m1 values, the nearest with ties to
the even code, scales by the exponent of the largest magnitude."""

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def pitch(k):
    return (k + 511) // 512 * 512


def scale_byte(top):
    """The scale byte of a block whose largest magnitude is `top`."""
    if not np.isfinite(top):
        return 255
    if top == 0:
        return 127
    return max(int(np.frexp(np.float64(top))[1]) - 1 - 2 + 127, 0)


def encode(v):
    """Codes of values already divided by their scale."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 6.0)
    hi = np.searchsorted(VALUES, a)
    lo = np.maximum(hi - 1, 0)
    below, above = a - VALUES[lo], VALUES[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 3)


def quantize(w):
    """(codes [n][pitch / 2], scales [n][pitch / 32]) of w [n][k]."""
    w = np.asarray(w, dtype=np.float64)
    n, k = w.shape
    kp = pitch(k)
    codes = np.zeros((n, kp), dtype=np.uint8)
    scales = np.full((n, kp // 32), 127, dtype=np.uint8)
    for i in range(n):
        for b in range((k + 31) // 32):
            t = w[i, 32 * b:32 * b + 32]
            top = np.nan if not np.all(np.isfinite(t)) else np.abs(t).max()
            s = scales[i, b] = scale_byte(top)
            if s != 255:
                codes[i, 32 * b:32 * b + len(t)] = encode(t * 2.0 ** (127 - int(s)))
    return codes[:, ::2] | codes[:, 1::2] << 4, scales


def values(codes, scales, k):
    """The values (float64) that codes stand for, [n][k]."""
    n = codes.shape[0]
    q = np.stack([codes & 15, codes >> 4], -1).reshape(n, -1)
    v = np.where(q >> 3, -1.0, 1.0) * VALUES[q & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * np.repeat(s, 32, axis=1))[:, :k]


def norm(s, weight, eps):
    """y of the sum s [rows][d]."""
    s = np.asarray(s, dtype=np.float64)
    r = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s * r * (1.0 if weight is None else weight.astype(np.float64))


def norm_backward(dy, s, weight, eps, dsum):
    """(ds, dweight)."""
    dy, s = dy.astype(np.float64), s.astype(np.float64)
    r = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    u = dy * (1.0 if weight is None else weight.astype(np.float64))
    ds = r * u - s * r ** 3 * (u * s).mean(1, keepdims=True)
    return ds + (0.0 if dsum is None else dsum.astype(np.float64)), (dy * s * r).sum(0)


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v < 0, e / (1 + e), 1 / (1 + e))


def gated(gate, up):
    return gate * sigmoid(gate) * up


def gated_backward(gate, up, dh):
    """(dgate, dup)."""
    t = sigmoid(gate)
    return dh * up * t * (1 + gate * (1 - t)), dh * gate * t
