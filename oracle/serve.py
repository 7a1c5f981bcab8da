"""Serving operators in 64 bits (oracle; test infrastructure only): e4m3 with block scales and
their product, the quantized cache.

The scales are part of the definition as 32-bit numbers (they are stored so), and so is the
reciprocal that the values are multiplied with; everything else is float64.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def e4m3_value(byte):
    """The values of e4m3 bytes: (-1)^s 2^(e - 7) (1 + m / 8), e = 0 subnormal, 0x7f NaN."""
    b = np.asarray(byte).astype(np.int64)
    s, e, m = b >> 7, (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    return np.where((b & 127) == 127, np.nan, np.where(s == 1, -v, v))


_TABLE = e4m3_value(np.arange(127))          # 0 .. 448, increasing
_MID = (_TABLE[1:] + _TABLE[:-1]) / 2


def e4m3_byte(v):
    """The byte of the nearest value (ties to the even byte), saturating; NaN for NaN or inf."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    i = np.searchsorted(_MID, a, side="left")        # a tie stays with the lower byte
    tie = (i < len(_MID)) & (a == _MID[np.minimum(i, len(_MID) - 1)])
    i = np.where(tie & (i % 2 == 1), i + 1, i)
    b = np.where(np.signbit(v), i + 128, i)
    return np.where(np.isfinite(v), b, 127).astype(np.uint8)


def _scale(amax):
    return np.maximum(np.float32(amax) / np.float32(E4M3_MAX), np.float32(SCALE_MIN))


def _reciprocal(s):
    return (np.float32(1.0) / s).astype(np.float64)


def fp8_quantize(X, block_rows: int):
    """(bytes, fp32 scales) of X (values of at most 32 bits) in blocks of block_rows x 128."""
    X = np.asarray(X, dtype=np.float64)
    rows, cols = X.shape
    R, C = -(-rows // block_rows), -(-cols // 128)
    scales = np.zeros((R, C), dtype=np.float32)
    codes = np.zeros((rows, cols), dtype=np.uint8)
    for i in range(R):
        for j in range(C):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            blk = X[at]
            fin = np.abs(blk[np.isfinite(blk)])
            s = _scale(fin.max() if fin.size else 0.0)
            scales[i, j] = s
            codes[at] = e4m3_byte(blk * _reciprocal(s))
    return codes, scales


def fp8_matmul(A, sA, B, sB):
    """(Y, sum of the magnitudes of the terms of each element) of e4m3 bytes and their scales."""
    a, b = e4m3_value(A), e4m3_value(B)
    Y = np.zeros((A.shape[0], B.shape[0]))
    M = np.zeros_like(Y)
    jb = np.arange(B.shape[0]) // 128
    for k in range(sA.shape[1]):
        at = np.s_[:, 128 * k:128 * (k + 1)]
        s = sA[:, k].astype(np.float64)[:, None] * sB[jb, k].astype(np.float64)[None, :]
        Y += a[at] @ b[at].T * s
        M += np.abs(a[at]) @ np.abs(b[at]).T * s
    return Y, M


def cache_quantize(X, bits, group: int):
    """Rows X (... x head_dim) in groups: dict of codes (one per value; e4m3 bytes where bits is
    None), scales (fp32), zeros and the values they stand for (fp64)."""
    X = np.asarray(X, dtype=np.float64)
    head = X.shape[:-1]
    x = X.reshape(*head, -1, group or X.shape[-1])
    if bits is None:
        fin = np.where(np.isfinite(x), np.abs(x), 0.0)
        s = _scale(fin.max(-1))
        c = e4m3_byte(x * _reciprocal(s)[..., None])
        z = np.zeros(s.shape, dtype=np.uint8)
        val = e4m3_value(c) * s.astype(np.float64)[..., None]
    else:
        maxq = 2 ** bits - 1
        bad = ~np.isfinite(x).all(-1)
        xs = np.where(bad[..., None], 0.0, x)
        mn, mx = np.minimum(xs.min(-1), 0.0), np.maximum(xs.max(-1), 0.0)
        flat = mn == mx
        mn, mx = np.where(flat, -1.0, mn), np.where(flat, 1.0, mx)
        with np.errstate(over="ignore"):
            rng = np.float32(mx) - np.float32(mn)
        bad |= ~np.isfinite(rng)
        rng = np.where(np.isfinite(rng), rng, np.float32(1.0))
        s = np.maximum(rng / np.float32(maxq), np.float32(SCALE_MIN))
        z = np.rint(-mn * maxq / (mx - mn))
        c = np.clip(np.rint(xs * _reciprocal(s)[..., None] + z[..., None]), 0, maxq)
        z = np.where(bad, 0, z).astype(np.uint8)
        c = np.where(bad[..., None], 0, c).astype(np.uint8)
        s = np.where(bad, np.float32(np.nan), s).astype(np.float32)
        val = (c.astype(np.float64) - z[..., None]) * s.astype(np.float64)[..., None]
    return dict(codes=c.reshape(X.shape), scales=s, zeros=z, values=val.reshape(X.shape))


def pack4(codes):
    """Two 4-bit codes per byte, the even one in the low half."""
    c = np.asarray(codes, dtype=np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)
