"""The 8-bit floating-point form in 64 bits, for the tests: codes, scales and
products from the definition, in numpy."""
import numpy as np

AMAX_FLOOR = 2.0 ** -90


def e4m3_table():
    """The value of every e4m3 bit pattern (NaN for the two NaN patterns)."""
    v = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v[b] = (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) * (-1 if s else 1)
        if e == 15 and m == 7:
            v[b] = np.nan
    return v


TABLE = e4m3_table()


def e4m3_round(q):
    """The e4m3 bit patterns nearest to q (64 bits, |q| <= 448 after
    saturation), ties to the even pattern, by search in the sorted values."""
    pos = TABLE[:127]                                   # 0 .. 448 ascending
    a = np.minimum(np.abs(q), 448.0)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    code = np.where(a == 0, 0, code)
    return (code | np.where(np.signbit(q), 128, 0)).astype(np.uint8)


def block_max(x, tall):
    m, d = x.shape
    p = np.pad(np.abs(x), ((0, -m % tall), (0, -d % 128)))
    return p.reshape(p.shape[0] // tall, tall, p.shape[1] // 128, 128).max(axis=(1, 3))


def spread(s, tall, m, d):
    return np.repeat(np.repeat(s, tall, 0), 128, 1)[:m, :d]


def quantize(x, tall):
    """x (64 bits) -> bit patterns, scales [row blocks, blocks] (fp32)."""
    a = np.maximum(block_max(x, tall), AMAX_FLOOR)
    s = (a.astype(np.float32) / np.float32(448)).astype(np.float32)
    return e4m3_round(x / spread(s.astype(np.float64), tall, *x.shape)), s


def values(codes, scales, tall):
    return TABLE[codes] * spread(scales.astype(np.float64), tall, *codes.shape)


def act(g, name):
    from scipy.special import expit, ndtr
    return g * expit(g) if name == "silu" else g * ndtr(g)
