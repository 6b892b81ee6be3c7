"""CPU oracle of the operators in include/snapkv_draft.h: fp64 numpy, one head at a time, from their
definitions. Test infrastructure only."""
from __future__ import annotations

import numpy as np

SMALLEST_STEP = 2.0 ** -80


def quantise(x):
    """Signs (-1, 1), magnitudes u [..., d] and steps h [...] of rows x [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.abs(x).max(-1)
        h = (top / 127.0).astype(np.float32).astype(np.float64)
        h = np.where(h < SMALLEST_STEP, 0.0, h)
        bad = ~np.isfinite(h)
        u = np.rint(np.abs(x) / np.where((h > 0) & ~bad, h, np.inf)[..., None])
    u = np.where(bad[..., None] | (h == 0)[..., None], 0, u).astype(np.int64)
    return np.where(np.signbit(x), -1, 1), u, np.where(bad, np.nan, h)


def codes(sign, u):
    return (u + np.where(sign < 0, 128, 0)).astype(np.uint8)


def values(code, h):
    """What codes uint8 [..., d] with steps [...] stand for."""
    code = np.asarray(code).astype(np.int64)
    return (code & 127) * np.where(code > 127, -1.0, 1.0) * np.asarray(h, dtype=np.float64)[..., None]


def attend(q, k, v, k_new=None, v_new=None, mask=None):
    """Tokens q [T, d] of one query head over the cached rows k, v [n, d] and the drafted ones [T, d] that mask [T, T] names.

    Returns out [T, d], lse [T], per-token bounds on the logits' terms [T], and sum p |v| [T, d]."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    T, d = q.shape
    out, lse, size, pv = np.zeros((T, d)), np.full(T, -np.inf), np.zeros(T), np.zeros((T, d))
    for t in range(T):
        kk, vv = k, v
        if k_new is not None:
            seen = np.asarray(mask[t], dtype=bool)
            kk = np.concatenate([k, np.asarray(k_new, dtype=np.float64)[seen]])
            vv = np.concatenate([v, np.asarray(v_new, dtype=np.float64)[seen]])
        if kk.shape[0] == 0:
            continue
        s = kk @ q[t] / np.sqrt(d)
        top = s.max()
        if top == -np.inf:
            continue
        p = np.exp(s - top)
        lse[t] = top + np.log(p.sum())
        p /= p.sum()
        out[t], pv[t] = p @ vv, p @ np.abs(vv)
        size[t] = (np.abs(kk) @ np.abs(q[t])).max() / np.sqrt(d)
    return out, lse, size, pv


def append(cache, new, pick, n, length):
    """One head's cache rows [cap, ...] after rows pick[:n] of new were appended at `length`."""
    res = np.array(cache)
    for i in range(n):
        res[length + i] = new[pick[i] if pick is not None else i]
    return res
