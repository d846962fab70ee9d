"""Oracle of the block-scaled e4m3 operators, in numpy, from their definition:
a block of 128 columns of a row (or 128 x 128 of a weight) has the scale
a / 448 with a = max(max |x|, 2^-100), and holds e4m3 numbers
q = round-half-even(RN32(x * RN32(448 / a))).  Products, norms and gates are
evaluated in 64 bits.

An e4m3 byte is sign | exponent (4 bits, bias 7) | mantissa (3 bits);
exponent 0 holds the subnormals m * 2^-9, and 0x7f / 0xff are the NaNs, so
the largest number is 0x7e = 448.
"""
from __future__ import annotations

import numpy as np

__all__ = ["E4M3_VALUES", "e4m3_decode", "e4m3_encode", "quantize_blocks", "quantize_weight_blocks",
           "spread_columns", "rms_norm64", "silu_mul64", "matmul64", "pack_weight"]

BLOCK = 128
_CODES = np.arange(127)
#: the 127 finite magnitudes in ascending order; the index is the byte
E4M3_VALUES = np.where(_CODES >> 3 == 0, (_CODES & 7) * 2.0 ** -9,
                       (1 + (_CODES & 7) / 8.0) * 2.0 ** ((_CODES >> 3) - 7.0))


def e4m3_decode(b):
    """bytes (uint8) -> float64 (NaN for 0x7f and 0xff)"""
    b = np.asarray(b, dtype=np.uint8)
    mag = np.concatenate([E4M3_VALUES, [np.nan]])[b & 0x7f]
    return np.where(b >> 7, -mag, mag)


def e4m3_encode(x):
    """numbers of magnitude below 464 (where 448 stops being the nearest) ->
    bytes, round to nearest, ties to the even byte; NaN -> a NaN byte"""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    mag = np.where(nan, 0.0, np.abs(x))
    assert np.all(mag < 464.0)
    hi = np.minimum(np.searchsorted(E4M3_VALUES, mag), 126)  # first value >= mag
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - E4M3_VALUES[lo], E4M3_VALUES[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(mag > 448.0, 126, code)
    code = np.where(nan, 127, code).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def _scales(amax):
    a = np.maximum(amax.astype(np.float32), np.float32(2.0 ** -100))
    return (a / np.float32(448.0)).astype(np.float32), (np.float32(448.0) / a).astype(np.float32)


def quantize_blocks(X):
    """X [M, K] (any float type that fp32 holds) -> (bytes [M, K], scales fp32
    [ceil(K/128), M]), bit for bit.  NaNs do not count for a block's maximum."""
    X = np.asarray(X).astype(np.float32)
    M, K = X.shape
    kb = -(-K // BLOCK)
    q = np.empty((M, K), np.uint8)
    s = np.empty((kb, M), np.float32)
    for b in range(kb):
        c = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        s[b], inv = _scales(np.fmax.reduce(np.abs(X[:, c]), axis=1, initial=0.0))
        with np.errstate(invalid="ignore"):
            q[:, c] = e4m3_encode(X[:, c] * inv[:, None])
    return q, s


def quantize_weight_blocks(W):
    """W [K, N] -> (bytes [N, K] row-major, scales fp32 [ceil(N/128), ceil(K/128)])"""
    Wt = np.ascontiguousarray(np.asarray(W).astype(np.float32).T)
    N, K = Wt.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    q = np.empty((N, K), np.uint8)
    s = np.empty((nb, kb), np.float32)
    for i in range(nb):
        for j in range(kb):
            t = Wt[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            s[i, j], inv = _scales(np.abs(t).max())
            q[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = e4m3_encode(t * inv)
    return q, s


def spread_columns(s, K):
    """scales [ceil(K/128), M] -> [M, K] float64, one per element"""
    return np.repeat(np.asarray(s, np.float64), BLOCK, axis=0)[:K].T


def rms_norm64(h, g, eps):
    h = np.asarray(h, np.float64)
    return h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(g, np.float64)


def silu_mul64(gate_up):
    gate_up = np.asarray(gate_up, np.float64)
    K = gate_up.shape[1] // 2
    g, u = gate_up[:, :K], gate_up[:, K:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def matmul64(xq, xs, wq, ws, bias=None):
    """bytes xq [M, K], wq [N, K] row-major with their scales -> (Y float64
    [M, N], the same sum over the absolute values, and over the groups of 8
    columns the largest |x| times the largest |w|, each at least the smallest
    normal number 2^-6)"""
    (M, K), N = xq.shape, wq.shape[0]
    xv, wv = e4m3_decode(xq), e4m3_decode(wq)
    sx = spread_columns(xs, K)
    sw = np.repeat(np.repeat(np.asarray(ws, np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]
    y, mag = (xv * sx) @ (wv * sw).T, np.abs(xv * sx) @ np.abs(wv * sw).T
    top = lambda v: np.maximum(np.abs(v).reshape(len(v), K // 8, 8).max(2), 2.0 ** -6)  # noqa: E731
    grain = (top(xv) * np.abs(sx[:, ::8])) @ (top(wv) * np.abs(sw[:, ::8])).T
    if bias is not None:
        b = np.asarray(bias, np.float64)
        y, mag = y + b, mag + np.abs(b)
    return y, mag, grain


def pack_weight(wq):
    """bytes [N, K] row-major -> the packed layout [N, roundup(K, 128)]: blocks
    of 16 rows x 128 columns, chunks of 16 columns first, then rows"""
    N, K = wq.shape
    Kp = -(-K // BLOCK) * BLOCK
    full = np.zeros((N, Kp), np.uint8)
    full[:, :K] = wq
    return np.ascontiguousarray(full.reshape(N // 16, 16, Kp // 128, 8, 16).transpose(0, 2, 3, 1, 4)).reshape(N, Kp)
