"""Bounds on the bf16 path of attn_extend and attn_decode_prefix that follow its
arithmetic term by term, for caches without rotations (identity matrices, where
the query rotation is exact), and an emulation of that arithmetic's roundings.

A score is s = scale * sum_d q_d k_d.  The kernels compute it from

* q as two fp16 values of a row scaled by a power of two: each component off by
  2^-22 of itself, or 2^-25 of a row whose largest is above 2^6 (2^-31 of it);
  before that one float32 rounding of q_d times the factor, itself two roundings;
* an INT2 key as its middle m (z + s, or z + rho s) and steps x_d = k_d - m,
  uniform steps exact, Lloyd-Max steps as a value and a residue that meets only
  q's high part (2^-22 for the residue's rounding, 2^-22 for q's low part); the
  middle as two fp16 values (2^-22 of it, 2^-25 of the scaled row) times the
  group's sum Q of the split q (float32, some 9 roundings; two fp16 values,
  2^-22); BF16 keys exact but for 2^-25 of the scaled row, where its small
  channels are subnormal.  A row is scaled by one half if its largest value is
  between 2^-2 and 2^14, else to just below 2^13;
* products summed by the tensor cores, M of them for 16 channels each, every one
  cutting the running sum off by 2^-24 of the magnitudes it has seen.
"""
import math

import numpy as np

from oracle import oscar_oracle as O

LM = float(np.float32(1.16))


def largest(c, cache, layer, role, b, h, T):
    """(rows [T][D], scale and zero of the INT2 ones, their range, largest value that a row's scaling goes by [T])."""
    X = O.dequant_history(c, cache, layer, role, b, h, T).astype(np.float64)
    m, sz, lo, hi = np.abs(X).max(1), None, c.sink, max(c.sink, T - c.recent)
    if hi > lo and not (role and c.flags & O.FLAG_V_BF16):
        sz = O.CacheView(c, cache, layer, role).sz[b, h, :hi - lo].astype(np.float64)
        span = 2 * LM + 1 if c.flags & O.FLAG_LLOYD_MAX else 3.0
        m[lo:hi] = np.maximum(np.abs(sz[..., 1]), np.abs(sz[..., 1] + span * sz[..., 0])).max(1)
    return X, sz, slice(lo, hi), m


def values(c, cache, layer, b, h, T):
    """Value rows [T][D] and what fp16's smallest number is in each [T]: 2^-25 of a row scaled to below 1, which rows with
    a largest value between 2^-8 and 2^12 are not."""
    V, _, _, m = largest(c, cache, layer, 1, b, h, T)
    e = np.floor(np.log2(np.where(m > 0, m, 1.0))) + 1
    return V, 2.0 ** -25 * 2.0 ** np.where((m == 0) | (m >= 2.0 ** -8) & (m < 2.0 ** 12), 0.0, np.clip(e, -60, 126))


def pieces(c, cache, layer, b, h, T):
    """Keys [T][D] of an INT2 / BF16 history as (middles [T][D/128], steps [T][D], INT2 scales [T][D/128], row factors [T]:
    the powers of two that undo the rows' scaling)."""
    K, sz, packed, m = largest(c, cache, layer, 0, b, h, T)
    mid, s = np.zeros((T, c.head_dim // 128)), np.zeros((T, c.head_dim // 128))
    if sz is not None:
        s[packed] = sz[..., 0]
        mid[packed] = sz[..., 1] + (LM if c.flags & O.FLAG_LLOYD_MAX else 1.0) * sz[..., 0]
    e = np.floor(np.log2(np.where(m > 0, m, 1.0))) + 1 - 13
    return mid, K - np.repeat(mid, 128, axis=1), s, np.where((m == 0) | (m >= 2.0 ** -2) & (m < 2.0 ** 14), 2.0, 2.0 ** e)


def score_bound(q, mid, steps, factor, scale, lm):
    """Bound on the error of every score of the query rows q [n][D]: [n][T]."""
    D = q.shape[1]
    aq, qs, qa = np.abs(q), np.abs(q.reshape(len(q), -1, 128).sum(-1)), np.abs(q).reshape(len(q), -1, 128).sum(-1)
    part = aq @ np.abs(steps).T
    middle = qs @ np.abs(mid).T
    products = D // 16 * (3 if lm else 2) + 1
    err = (2.0 ** -22 + (2.0 ** -21 if lm else 0)) * part
    err += 2.0 ** -31 * aq.max(1)[:, None] * np.abs(steps).sum(1)
    err += 3 * 2.0 ** -24 * (part + middle) + 2.0 ** -25 * aq.sum(1)[:, None] * factor
    err += 2 * 2.0 ** -22 * middle + 2.0 ** -25 * qs.sum(1)[:, None] * factor + 10 * 2.0 ** -24 * (qa @ np.abs(mid).T)
    err += products * 2.0 ** -24 * (part + middle)
    return scale * err


def attend(q, mid, steps, factor, V, floor, hidden, scale, lm):
    """Query rows q [n][D] over one history: (out [n][D], lse [n], bounds of out per element, bounds of lse).

    With scores off by e_t the log-sum-exp moves by sum p_t e_t at most (p at a point between, within exp(2 max e) of the
    exact one), and a probability by e_t plus that of itself.  P and the value rows are rounded to fp16, 2^-11 each (a
    Lloyd-Max value's unit and middle as well, each at most as large as the largest value of its row), small channels of a
    value row to its `floor` (up to three roundings with Lloyd-Max levels); the float32 steps
    are the exponential's and the logarithm's 2^-22, the scores less their reference, sums over tiles and shares."""
    T = len(mid)
    K = steps + np.repeat(mid, 128, axis=1)
    s = scale * (q @ K.T)
    s[hidden] = -np.inf
    top = s.max(1)
    p = np.exp(s - top[:, None])
    l = p.sum(1)
    p /= l[:, None]
    e = score_bound(q, mid, steps, factor, scale, lm)
    e[hidden] = 0
    mean = (p * e).sum(1) * np.exp(2 * e.max(1))
    lse = top + np.log(l)
    small = 2.0 ** -21 + (T / 128 + 80) * 2.0 ** -24
    lb = mean + small + 8 * 2.0 ** -24 * (np.abs(lse) + 16)
    out = p @ V
    size = np.abs(V) if not lm else np.abs(V).max(1, keepdims=True) * np.ones_like(V)
    rel = (2 + (2 if lm else 0)) * 2.0 ** -11 + 2 * small + 8 * 2.0 ** -24 * (np.abs(lse) + 16)
    ob = (p * (e + mean[:, None] + rel[:, None])) @ size + 3 * (p @ floor)[:, None] + 2.0 ** -33 * size.sum(0) + 2.0 ** -8 * np.abs(out) * 1.01
    return out, lse, ob * 1.01, lb


def f16(x):
    return np.asarray(x, np.float64).astype(np.float16).astype(np.float64)


def emulated_scores(q, mid, steps, s, scale, lm, drop=""):
    """The scores with the operands rounded as the kernels round them, everything else exact; `drop` leaves a part out:
    "q": the query's low part, "middle": the middles' and the sums' low parts, "residue": the Lloyd-Max residues."""
    q = (q * np.float32(scale * math.log2(math.e))).astype(np.float32).astype(np.float64)  # rotated queries are in log2 units
    f = 2.0 ** (6 - np.floor(np.log2(np.abs(q).max(1, keepdims=True))))
    x = q * f
    hi = f16(x)
    lo = np.zeros_like(hi) if drop == "q" else f16(x - hi)
    g = lambda y: y.reshape(len(y), -1, 128)
    two = lambda y: f16(y) + (0 if drop == "middle" else f16(y - f16(y)))
    if lm:
        w = np.repeat(s, 128, axis=1) > 0
        value = np.where(w, f16(steps * 0.5), steps * 0.5)
        rest = np.where(w, f16(steps * 0.5 - value), 0) if drop != "residue" else 0 * value
        total = (hi + lo) @ value.T + hi @ rest.T
    else:
        total = (hi + lo) @ f16(steps * 0.5).T
    total = total + two(g(hi + lo).sum(-1)) @ two(mid * 0.5).T
    return total * 2 / f * math.log(2.0)
