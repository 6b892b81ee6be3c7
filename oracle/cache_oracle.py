"""CPU oracle of the operators in include/snapkv_cache.h: fp64 numpy, one head at a time, from their
definitions. Test infrastructure only."""
from __future__ import annotations

import numpy as np

GROUP = 64
SIGN_BIT = (15, 14, 7, 6)
MAG_BIT = (3, 0, 11, 8)


def bf16(x):
    """x rounded to bf16 (through fp32), as float64."""
    x = np.asarray(x, dtype=np.float32)
    bits = x.view(np.uint32).astype(np.uint64)
    out = ((bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), out).astype(np.float64)


def quantise(x):
    """Level numbers u [..., d], h and z [..., d / 64] of rows x [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(invalid="ignore", over="ignore"):
        hi, lo = g.max(-1), g.min(-1)
        h, z = bf16((hi - lo) / 30.0), bf16((hi + lo) / 2.0)
        h = np.where(h < 2.0 ** -126, 0.0, h)
        bad = ~(np.isfinite(h) & np.isfinite(z))
        step = np.where((h > 0) & ~bad, 2.0 * h, np.inf)
        u = np.rint(np.clip((g - np.where(bad, 0.0, z)[..., None]) / step[..., None] + 7.5, 0, 15))
    u = np.where((h == 0)[..., None] | bad[..., None], 8, u).astype(np.int64)
    return u.reshape(x.shape), np.where(bad, np.nan, h), np.where(bad, np.nan, z)


def pack(u):
    """Level numbers [..., d] as codes uint8 [..., d / 2]."""
    d = u.shape[-1]
    ng = d // GROUP
    words = np.zeros((*u.shape[:-1], d // 8), dtype=np.uint32)
    for c in range(d):
        e, j = c % 8, (c % 8) // 2
        t = 2 * u[..., c] - 15
        field = ((t < 0).astype(np.uint32) << SIGN_BIT[j]) | (((np.abs(t) - 1) // 2).astype(np.uint32) << MAG_BIT[j])
        words[..., ng * ((c % GROUP) // 8) + c // GROUP] |= field << np.uint32(16 * (e % 2))
    return words.view(np.uint8).reshape(*u.shape[:-1], d // 2)


def values(u, h, z):
    """What levels u with (h, z) stand for."""
    t = (2.0 * u - 15.0).reshape(*u.shape[:-1], -1, GROUP)
    return (z[..., None] + h[..., None] * t).reshape(u.shape)


def magnitudes(u, h, z):
    """|z| + |h t|: what sums over a 4-bit row's parts are bounded by."""
    t = np.abs(2.0 * u - 15.0).reshape(*u.shape[:-1], -1, GROUP)
    return (np.abs(z)[..., None] + np.abs(h)[..., None] * t).reshape(u.shape)


def attend(q, k, v, k_size=None, v_size=None):
    """One query over the rows k, v [n, d]: (out [d], weights [n], per-row logit bound, per-channel bound).

    The bounds are sums of magnitudes, for tolerances: of the largest logit's terms, and sum p |v|."""
    d = q.shape[-1]
    if k.shape[0] == 0:
        return np.zeros(d), np.zeros(0), 0.0, np.zeros(d)
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    s = k @ q / np.sqrt(d)
    p = np.exp(s - s.max())
    p /= p.sum()
    size = ((np.abs(k) if k_size is None else k_size) @ np.abs(q)).max() / np.sqrt(d)
    return p @ v, p, size, p @ (np.abs(v) if v_size is None else v_size)


def evict_slots(score, length, keep, recent):
    """Source slot of each of the first min(length, keep + recent) slots of one head."""
    left = keep + recent
    if length <= left:
        return np.arange(length)
    n = length - recent
    key = np.where(np.isnan(score[:n]), -np.inf, score[:n])
    # NaN below everything, -inf included
    order = sorted(range(n), key=lambda r: (np.isnan(score[r]), -key[r], r))
    stays = np.zeros(n, dtype=bool)
    stays[order[:keep]] = True
    src = np.arange(left)
    movers = [r for r in range(keep, n) if stays[r]]
    for slot in range(keep):
        if not stays[slot]:
            src[slot] = movers.pop(0)
    src[keep:] = np.arange(n, length)
    return src
