"""Plain 64-bit reference of the 8-bit checkpoint format (test infrastructure).

Values in and out are float64 numpy arrays; codes and exponent bytes are laid
out as the library's buffer. Rounding goes by the table of the format's values,
ties to the even code.
"""
import numpy as np

E4M3, INT8 = 2, 3
TOP = {E4M3: 448.0, INT8: 127.0}


def table(fmt):
    """Non-negative values by code."""
    if fmt == INT8:
        return np.arange(128, dtype=np.float64)
    c = np.arange(127)
    ex, fr = c >> 3, c & 7
    return np.where(ex > 0, (1 + fr / 8) * 2.0 ** (ex - 7.0), fr * 2.0 ** -9)


def pitch(cols):
    return -(-cols // 32) * 32


def nbytes(rows, cols):
    return rows * (pitch(cols) + pitch(cols) // 32)


def exponent(amax, fmt):
    """Smallest e >= -124 with amax <= TOP * 2^e (exact in float64)."""
    m, k = np.frexp(amax / TOP[fmt])  # the division by 7 * 2^6 or 127 may round: mend below
    e = k - (m == 0.5)
    e = np.where(amax <= TOP[fmt] * np.exp2(e - 1.0), e - 1, e)
    e = np.where(amax > TOP[fmt] * np.exp2(e * 1.0), e + 1, e)
    return np.where(amax == 0, -124, np.maximum(e, -124)).astype(np.int64)


def pack(x, fmt):
    """(codes uint8 [rows, P], exponent bytes uint8 [rows, P / 32])."""
    rows, cols = x.shape
    b = np.zeros((rows, pitch(cols)))
    b[:, :cols] = x
    b = b.reshape(rows, -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = exponent(amax, fmt)
    t = table(fmt)
    a = np.abs(b) * np.exp2(-e.astype(np.float64))[..., None]
    mid = (t[1:] + t[:-1]) / 2
    at = np.searchsorted(mid, a, side="left")
    tie = a == mid[np.minimum(at, mid.size - 1)]
    at = at + (tie & (at % 2 == 1))
    # the largest code whose value stays finite in fp32
    most = np.searchsorted(t, 2.0 ** 128 / np.exp2(e.astype(np.float64)), side="left") - 1
    at = np.minimum(at, most[..., None])
    neg = np.signbit(b)
    codes = np.where(neg, at + 128, at) if fmt == E4M3 else np.where(neg, -at, at) & 255
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(rows, -1), np.where(bad, 255, e + 127).astype(np.uint8)


def unpack(codes, exps, cols, fmt):
    rows = codes.shape[0]
    c = codes.reshape(rows, -1, 32).astype(np.int64)
    if fmt == INT8:
        v = np.where(c > 127, c - 256, c).astype(np.float64)
    else:
        v = table(fmt)[np.minimum(c & 127, 126)]
        v = np.where(c & 128, -v, v)
    s = np.where(exps == 255, np.nan, np.exp2(exps.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(rows, -1)[:, :cols]


def buffer(codes, exps):
    return np.concatenate([codes.reshape(-1), exps.reshape(-1)])


def split(buf, rows, cols):
    p = pitch(cols)
    return buf[: rows * p].reshape(rows, p), buf[rows * p: nbytes(rows, cols)].reshape(rows, p // 32)


def held(x, fmt):
    return unpack(*pack(x, fmt), x.shape[1], fmt)
