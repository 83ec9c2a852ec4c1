"""Plain numpy definitions of the 8-bit form of rows and weights, of its norm and products, and of log probabilities.

Everything is written from the definitions, in float64: one group, one row at a time.
"""
from __future__ import annotations

import numpy as np

from .q4 import bf16_f64, bf16_round

GROUP = 128
LARGEST = 448.0


def code_values():
    """What the bytes 0..127 of the 8-bit format stand for: 4 bits of exponent, 3 of significand; the last is NaN."""
    v = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)]
    return np.array(v[:127] + [np.nan])


VALUES = code_values()


def nearest(q):
    """q [..] -> bytes: the nearest value, the even byte of two that are as near, the largest beyond it."""
    q = np.asarray(q, np.float64)
    a = np.minimum(np.abs(q), LARGEST)
    hi = np.clip(np.searchsorted(VALUES[:127], a), 1, 126)
    lo = hi - 1
    up, down = VALUES[hi] - a, a - VALUES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def scale(amax):
    """The smallest power of two, 2^-126 at least, that 448 times is not below amax."""
    if not np.isfinite(amax):
        return np.nan
    s = 2.0 ** -126
    while LARGEST * s < amax:
        s *= 2
    return s


def groups(n):
    return -(-n // GROUP)


def quantise(x, by=1):
    """x [R, C] float64 -> bytes [R, C], scales [ceil(R / by), groups] float64; by: rows of a scale, 1 or 128.  A group
    with a NaN or an infinity has a scale of NaN (its bytes are whatever they are: 0 here)."""
    R, C = x.shape
    codes = np.zeros((R, C), np.uint8)
    scales = np.zeros((-(-R // by), groups(C)))
    for i in range(scales.shape[0]):
        for g in range(scales.shape[1]):
            at = np.s_[i * by:(i + 1) * by, g * GROUP:(g + 1) * GROUP]
            part = x[at]
            s = scale(np.abs(part).max() if np.isfinite(part).all() else np.nan)
            scales[i, g] = s
            if np.isfinite(s):
                codes[at] = nearest(part / s)
    return codes, scales


def spread(scales, R, C):
    """Scales of rows [R, groups] or of a weight [groups, groups], one a value [R, C]."""
    by = 1 if scales.shape[0] == R else GROUP
    return np.repeat(np.repeat(scales, by, 0)[:R], GROUP, 1)[:, :C]


def value(codes, scales):
    v = VALUES[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    return v * spread(np.asarray(scales, np.float64), *codes.shape)


def rmsnorm(x, y=None, gain=None, eps=1e-6):
    """bf16 bits x, y [T, H], gain [H] -> (bits of x + y, the normalised rows in float64)."""
    s = x if y is None else bf16_round(bf16_f64(x) + bf16_f64(y))
    f = bf16_f64(s)
    h = f / np.sqrt((f * f).mean(1, keepdims=True) + eps)
    return s, h if gain is None else h * bf16_f64(gain)


def matmul(xc, xs, wc, ws):
    """(the product in float64, the sum of its terms' sizes)."""
    x, w = value(xc, xs), value(wc, ws)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def logprobs(logits, tokens, n):
    """logits [R, V] float64 -> (logprob [R], entropy [R], ids [R, n], their log probabilities [R, n])."""
    R, V = logits.shape
    lp, ent = np.zeros(R), np.zeros(R)
    ids, tops = np.full((R, n), -1, np.int32), np.full((R, n), -np.inf)
    for r in range(R):
        x = logits[r]
        k = min(n, V)
        if np.isnan(x).any() or (x == np.inf).any():
            lp[r] = 0.0 if tokens[r] == -1 else np.nan
            ent[r], tops[r] = np.nan, np.nan
            continue
        order = sorted(range(V), key=lambda v: (-x[v], v))[:k] if V <= 64 else np.lexsort((np.arange(V), -x))[:k]
        ids[r, :k] = order
        m = x.max()
        if m == -np.inf:
            lp[r] = 0.0 if tokens[r] == -1 else -np.inf
            continue
        e = np.exp(x - m)
        log_s = np.log(e.sum())
        logp = x - m - log_s
        p = np.exp(logp)
        ent[r] = -(p[p > 0] * logp[p > 0]).sum()
        tops[r, :k] = logp[ids[r, :k]]
        lp[r] = 0.0 if tokens[r] == -1 else logp[tokens[r]]
    return lp, ent, ids, tops
