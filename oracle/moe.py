"""Oracle of the mixture-of-experts operators and of the sandwich norm, in
numpy and 64 bits, from their definitions."""
from __future__ import annotations

import numpy as np

from .fp8_block import BLOCK, e4m3_decode, rms_norm64, silu_mul64

__all__ = ["sandwich64", "route64", "weight64", "moe64"]


def sandwich64(x, residual, post, pre, gate, alpha, eps):
    """(h, y, z): gate [G, K] or None, G dividing the rows"""
    z = rms_norm64(x, post, eps)
    if gate is not None:
        z = z * np.repeat(np.asarray(gate, np.float64), len(z) // len(gate), 0)
    h = alpha * np.asarray(residual, np.float64) + z
    return h, rms_norm64(h, pre, eps), z


def route64(x, w, top_k, normalize):
    """(experts, weights): descending logits, ties and NaNs (which rank with
    -inf) to the lower index"""
    with np.errstate(invalid="ignore", over="ignore"):
        logits = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
        key = np.where(np.isnan(logits), -np.inf, logits)
        experts = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
        p = np.exp(logits - key.max(1, keepdims=True))
        p = p / p.sum(1, keepdims=True)
        weights = np.take_along_axis(p, experts, 1)
        if normalize:
            weights = weights / weights.sum(1, keepdims=True)
    return experts, weights


def weight64(q, s):
    """bytes [N, K] with scales [ceil(N/128), ceil(K/128)] -> float64"""
    N, K = q.shape
    return e4m3_decode(q) * np.repeat(np.repeat(np.asarray(s, np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]


def moe64(x, experts, weights, up, up_s, down, down_s, sums):
    """(y, tol): bytes up [E, 2I, K], down [E, K, I]; tol bounds the error of an
    fp32 evaluation whose two products add within sums[0] and sums[1] of the sum
    of their terms' magnitudes, with the gated product between them within 8 half
    steps of 2^-24 of its formula and then held to 2^-17."""
    x = np.asarray(x, np.float64)
    y, tol = np.zeros((2, *x.shape))
    E, I2, _ = up.shape
    for e in range(E):
        m, j = np.nonzero(experts == e)
        if not len(m):
            continue
        wu, wd = weight64(up[e], up_s[e]), weight64(down[e], down_s[e])
        gu = x[m] @ wu.T
        err = sums[0] * (np.abs(x[m]) @ np.abs(wu).T)
        g, u, dg, du = gu[:, :I2 // 2], gu[:, I2 // 2:], err[:, :I2 // 2], err[:, I2 // 2:]
        a = silu_mul64(gu)
        silu = silu_mul64(np.concatenate([g, np.ones_like(g)], 1))
        # |silu'| <= 1.1
        da = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du
        da = da + (8 * 2.0 ** -24 + 2.0 ** -17) * (np.abs(a) + da)
        p = weights[m, j].astype(np.float64)[:, None]
        np.add.at(y, m, p * (a @ wd.T))
        np.add.at(tol, m, np.abs(p) * (da @ np.abs(wd).T + (sums[1] + 2.0 ** -23) * ((np.abs(a) + da) @ np.abs(wd).T)))
    # the pairs' sum: one half step each of what they come to
    return y, tol + experts.shape[1] * 2.0 ** -23 * (np.abs(y) + tol)
