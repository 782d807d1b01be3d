"""Plain 64-bit reference of the packed formats beside ckpt_ref's: 4-bit blocks
(e2m1), and matrices of any of the three (test infrastructure)."""
import numpy as np

import ckpt_ref as ref

E4M3, INT8, E2M1 = 2, 3, 4
TABLE = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def row_bytes(cols, fmt):
    return ref.pitch(cols) // 32 * (17 if fmt == E2M1 else 33)


def nbytes(rows, cols, fmt):
    return rows * row_bytes(cols, fmt)


def exponent(amax):
    """Smallest e >= -124 with amax <= 6 * 2^e."""
    m, k = np.frexp(amax)                     # amax = m 2^k, m in [1/2, 1); 6 2^e = 3/4 2^(e + 3)
    e = k - 3 + (m > 0.75)
    return np.where(amax == 0, -124, np.maximum(e, -124)).astype(np.int64)


def pack(x, fmt):
    """The buffer of fp64 x: codes, then exponent bytes."""
    if fmt != E2M1:
        return ref.buffer(*ref.pack(x, fmt))
    rows, cols = x.shape
    b = np.zeros((rows, ref.pitch(cols)))
    b[:, :cols] = x
    b = b.reshape(rows, -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = exponent(np.abs(b).max(-1))
    a = np.abs(b) * np.exp2(-e.astype(np.float64))[..., None]
    mid = (TABLE[1:] + TABLE[:-1]) / 2
    at = np.searchsorted(mid, a, side="left")
    at = at + ((a == mid[np.minimum(at, 6)]) & (at % 2 == 1))
    # the largest code whose value stays finite in fp32
    most = np.searchsorted(TABLE, 2.0 ** 128 / np.exp2(e.astype(np.float64)), side="left") - 1
    at = np.minimum(at, most[..., None])
    codes = np.where(bad[..., None], 0, np.where(np.signbit(b), at + 8, at)).astype(np.uint8).reshape(rows, -1)
    return ref.buffer(codes[:, ::2] | codes[:, 1::2] << 4, np.where(bad, 255, e + 127).astype(np.uint8))


def unpack(buf, rows, cols, fmt):
    p = ref.pitch(cols)
    if fmt != E2M1:
        return ref.unpack(*ref.split(buf, rows, cols), cols, fmt)
    n = rows * p // 2
    c = np.stack([buf[:n] & 15, buf[:n] >> 4], -1).reshape(rows, -1, 32).astype(np.int64)
    v = np.where(c & 8, -TABLE[c & 7], TABLE[c & 7])
    exps = buf[n:n + rows * p // 32].reshape(rows, -1)
    s = np.where(exps == 255, np.nan, np.exp2(exps.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(rows, -1)[:, :cols]


def held(x, fmt):
    return unpack(pack(x, fmt), *x.shape, fmt)
