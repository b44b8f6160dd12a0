"""Block-scaled e4m3 codes and tokens sorted by expert, on the CPU.

Written from the definitions: a table of the e4m3 values, nearest value with
ties to the even code, scales as one fp32 division, sums in 64 bits, loops over
slots and experts.
"""

import numpy as np

BLOCK = 128
TOP = 448.0


def _value(code):
    """The value of a non-negative e4m3 code: exponent bias 7, 3 mantissa bits."""
    e, m = code >> 3, code & 7
    return m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)


#: values of the codes 0 .. 126 (127 is not a number)
VALUES = np.array([_value(c) for c in range(127)])


def encode(v):
    """Codes (uint8) of fp32 values: clipped to +-448, nearest, ties to even."""
    v = np.asarray(v, dtype=np.float32).astype(np.float64)
    a = np.minimum(np.abs(v), TOP)
    hi = np.searchsorted(VALUES, a)               # first value >= a
    lo = np.maximum(hi - 1, 0)
    below, above = a - VALUES[lo], VALUES[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return code | (np.signbit(v).astype(np.uint8) << 7)


def decode(codes):
    """Values (float64) of codes."""
    codes = np.asarray(codes, dtype=np.uint8)
    v = VALUES[codes & 127]
    return np.where(codes >> 7, -v, v)


def pitch(k):
    return (k + BLOCK - 1) // BLOCK * BLOCK


def quantize(w, block_rows):
    """(codes [n][pitch], scales fp32) of fp32 values w [n][k]."""
    w = np.asarray(w, dtype=np.float32)
    n, k = w.shape
    kp = pitch(k)
    nb = (n + block_rows - 1) // block_rows
    codes = np.zeros((n, kp), dtype=np.uint8)
    scales = np.ones((nb, kp // BLOCK), dtype=np.float32)
    for i in range(nb):
        rows = slice(i * block_rows, min(n, (i + 1) * block_rows))
        for b in range(kp // BLOCK):
            cols = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
            t = w[rows, cols]
            s = np.float32(np.abs(t).max()) / np.float32(TOP)
            s = np.float32(1.0) if s == 0 else s
            scales[i, b] = s
            with np.errstate(over="ignore"):
                codes[rows, cols] = encode(t / s)
    return codes, scales


def values(codes, scales, block_rows, k):
    """The values (float64, unrounded) that codes stand for, [n][k]."""
    n = codes.shape[0]
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, axis=1), block_rows, axis=0)[:n]
    return (decode(codes) * s)[:, :k]


def swiglu(h):
    """silu(gate) * up of h [rows][2 f] in 64 bits."""
    h = np.asarray(h, dtype=np.float64)
    f = h.shape[1] // 2
    with np.errstate(over="ignore"):
        return h[:, :f] / (1.0 + np.exp(-h[:, :f])) * h[:, f:]


def sort(ids, experts):
    """(pos, order, offsets) by walking the slots expert by expert."""
    flat = np.asarray(ids).reshape(-1)
    pos = np.full(flat.size, -1, dtype=np.int32)
    order = np.full(flat.size, -1, dtype=np.int32)
    offsets = np.zeros(experts + 1, dtype=np.int32)
    row = 0
    for e in range(experts):
        offsets[e] = row
        for slot in np.nonzero(flat == e)[0]:
            pos[slot] = row
            order[row] = slot
            row += 1
    offsets[experts] = row
    return pos.reshape(np.shape(ids)), order, offsets


def combine(ys, pos, weights):
    """y [t][d] in 64 bits."""
    t, topk = pos.shape
    y = np.zeros((t, ys.shape[1]))
    for i in range(t):
        for j in range(topk):
            if 0 <= pos[i, j] < ys.shape[0]:
                w = 1.0 if weights is None else float(weights[i, j])
                y[i] += w * ys[pos[i, j]].astype(np.float64)
    return y


def combine_backward(dy, ys, pos, weights, dys):
    """(dys, dweights) in 64 bits; `dys` holds what rows without a slot keep."""
    t, topk = pos.shape
    dys = np.array(dys, dtype=np.float64)
    dw = np.zeros((t, topk))
    for i in range(t):
        for j in range(topk):
            p = pos[i, j]
            if 0 <= p < ys.shape[0]:
                w = 1.0 if weights is None else float(weights[i, j])
                dys[p] = w * dy[i].astype(np.float64)
                dw[i, j] = dy[i].astype(np.float64) @ ys[p].astype(np.float64)
    return dys, dw
