"""Block-scaled e4m3 in 64 bits, for the tests of the 8-bit expert products.

Plain numpy from the definitions: the e4m3 grid (4 exponent bits, bias 7, 3
mantissa bits, largest value 448, smallest step 2^-9), round to nearest even,
and power-of-two block scales.
"""
import numpy as np

BLOCK = 128
U32 = 2.0 ** -24   # half a step of fp32
UBF = 2.0 ** -8    # half a step of bf16


def e4m3_round(v):
    """The e4m3 value nearest v (ties to even), saturating at 448."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(v)))
    e = np.where(np.isfinite(e), np.maximum(e, -6), -6)
    step = 2.0 ** (e - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def scale_of(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    amax = np.maximum(np.asarray(amax, dtype=np.float64), 448.0 * 2.0 ** -126)
    m, x = np.frexp(amax)                    # amax = m 2^x, 1/2 <= m < 1; 448 = 7/8 2^9
    return 2.0 ** (x - 9 + (m > 0.875))


def _padded(x, axis):
    pad = [(0, 0)] * x.ndim
    pad[axis] = (0, -x.shape[axis] % BLOCK)
    return np.pad(x, pad)


def quantize_rows(x):
    """(q values [rows, cols], scales [ceil(cols / 128), rows])."""
    x = np.asarray(x, dtype=np.float64)
    b = _padded(x, 1).reshape(x.shape[0], -1, BLOCK)
    s = scale_of(np.abs(b).max(2))
    q = e4m3_round(b / s[:, :, None]).reshape(x.shape[0], -1)[:, :x.shape[1]]
    return q, s.T.copy()


def quantize_weights(W, transpose=False):
    W = np.asarray(W, dtype=np.float64)
    E, R, C = W.shape
    b = _padded(_padded(W, 1), 2)
    b = b.reshape(E, b.shape[1] // BLOCK, BLOCK, b.shape[2] // BLOCK, BLOCK)
    s = scale_of(np.abs(b).max((2, 4)))
    q = e4m3_round(b / s[:, :, None, :, None]).reshape(E, b.shape[1] * BLOCK, -1)[:, :R, :C]
    return (q.transpose(0, 2, 1).copy(), s.transpose(0, 2, 1).copy()) if transpose else (q, s)


def row_values(q, s):
    return q * np.repeat(s.T, BLOCK, 1)[:, :q.shape[1]]


def weight_values(q, s):
    return q * np.repeat(np.repeat(s, BLOCK, 1)[:, :q.shape[1]], BLOCK, 2)[:, :, :q.shape[2]]


def product(x, W, offsets):
    """(y, bound): the ragged grouped product of values in 64 bits, and a
    bound on the error of sums in fp32: every one of a row's additions (127
    inside a block, one per block, the scale's product) is off by at most a
    whole step (2^-23, allowing truncation) of a partial sum that the sum of
    the terms' sizes bounds."""
    y = np.zeros((x.shape[0], W.shape[1]))
    size = np.zeros_like(y)
    for e in range(W.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        y[r] = x[r] @ W[e].T
        size[r] = np.abs(x[r]) @ np.abs(W[e]).T
    blocks = -(-x.shape[1] // BLOCK)
    return y, (BLOCK + blocks + 4) * 2 * U32 * size


def row_expert(offsets, rows):
    return np.clip(np.searchsorted(offsets, np.arange(rows), side="right") - 1, 0, len(offsets) - 2)


def _spread(h, d):
    """Quantised values of h and how far they can lie apart when h is known
    to within d: every combination of the ends of its interval and of its
    block's scale."""
    rows, cols = h.shape
    q, s = quantize_rows(h)
    mid = row_values(q, s)
    lo, hi = mid.copy(), mid.copy()
    amax = lambda v: np.abs(_padded(v, 1)).reshape(rows, -1, BLOCK).max(2)  # noqa: E731
    for a in (np.maximum(np.abs(h) - d, 0), np.abs(h) + d):
        sc = np.repeat(scale_of(amax(a)), BLOCK, 1)[:, :cols]
        for v in (h - d, h, h + d):
            x = e4m3_round(v / sc) * sc
            lo, hi = np.minimum(lo, x), np.maximum(hi, x)
    return mid, hi - lo


def ffn(x, offsets, W1, W2, act, W3=None, b1=None, b2=None):
    """(y, bound) of the expert FFN on weight values (already dequantised):
    x and h quantised by rows; the bound follows the fp32 error of the first
    products through the activation, lets a hidden value that lies within it
    of a rounding border fall to either side, and adds the second product's
    error and the rounding of y to bf16."""
    from scipy.special import ndtr
    xv = row_values(*quantize_rows(x))
    ex = row_expert(offsets, x.shape[0])
    g, dg = product(xv, W1, offsets)
    if act == "swiglu":
        u, du = product(xv, W3, offsets)
        silu = g / (1.0 + np.exp(-g))
        h = silu * u
        # |silu'| < 1.1; the special-function silu is good to 4e-6
        d = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 4e-6 * np.abs(h) + 2 * U32 * np.abs(h)
    else:
        if b1 is not None:
            g = g + b1[ex]
            dg = dg + U32 * np.abs(g)
        h = g * ndtr(g)
        d = 1.13 * dg + 4.2e-7 + 2 * U32 * np.abs(h)  # |gelu'| < 1.13; the approximation's own error
    hv, dh = _spread(h, d)
    y, dy = product(hv, W2, offsets)
    dy = dy + product(dh, np.abs(W2), offsets)[0]
    if b2 is not None:
        y = y + b2[ex]
        dy = dy + U32 * np.abs(y)
    return y, dy + UBF * (np.abs(y) + dy)
