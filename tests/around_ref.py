"""Plain 64-bit forms of qk_norm_rope, attn_prompt, attn_mass and kv_evict, and how far float32 / bf16 arithmetic may be
from them (bounds per element, from the operands)."""
import math

import numpy as np

from oracle import oscar_oracle as O
from tests.rows_ref import rows64

F32, BF16 = 2.0 ** -24, 2.0 ** -8  # half a step of a rounding, relative


def norm_rope(x, w, eps, positions, inv_freq, interleaved, fp32):
    """x [n][heads][D]: (y, bound).  Float32: D squares added up, root, quotient and two products, relative
    (D / 2 + 6) 2^-24; an angle's last bit 2^-24 half turns, i.e. 2^-22.3 rad, sine and cosine 2 ulp: 2^-21 of |a| + |b| in
    all; one rounding to the output's type."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    size = np.abs(y)
    r = 0 if inv_freq is None else 2 * len(inv_freq)
    if r:
        phi = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
        i = np.arange(r // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = size[..., b] = np.abs(ya) + np.abs(yb)
    return y, size * ((D / 2 + 10) * F32 + 2.0 ** -21) + np.abs(y) * (F32 if fp32 else BF16) + 1e-37


def prompt(q, k, v, lens, first, scale, exact):
    """q [n][Hq][D], k, v [n][Hkv][D]; sequence b at rows first[b] .. + lens[b] - 1: (out, lse, bounds of both).
    exact: everything in float32.  Else scores are float32 sums on the tensor cores, which cut off (2^-23 of the magnitudes
    per step), probabilities are rounded to bf16 (2^-8), as is the output."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.full(q.shape, 7.0), np.full((n, Hq), 7.0)
    ob, lb = np.full(q.shape, 1e-30), np.full((n, Hq), 1e-30)
    for f, T in zip(first, lens):
        at = slice(f, f + T)
        hidden = np.triu(np.ones((T, T), bool), 1)
        for h in range(Hq):
            Q, K, V = (np.asarray(x, np.float64) for x in (q[at, h], k[at, h // G], v[at, h // G]))
            s = np.where(hidden, -np.inf, Q @ K.T * scale)
            size = np.where(hidden, 0, np.abs(Q) @ np.abs(K).T * scale).max(1, initial=0.0)
            ds = size * (D + 8) * (2 * F32 if exact else 4 * F32) + 1e-7
            m = s.max(1, initial=-np.inf, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p /= l
            out[at, h] = p @ V
            lse[at, h] = (m + np.log(l))[:, 0]
            rel = (2 * ds + (T + 64) * 2 * F32 + (0 if exact else BF16))[:, None]
            ob[at, h] = rel * (p @ np.abs(V))
            lb[at, h] = ds + (T + 64) * F32 + 4 * F32 * np.abs(lse[at, h])
    return out, lse, ob, lb


def check(name, got, want, bound):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all(), f"{name}: not finite at {np.argwhere(~np.isfinite(got))[:4].tolist()}"
    err = np.abs(got - want)
    bad = np.argwhere(err > bound)
    assert bad.size == 0, (f"{name}: {len(bad)} of {err.size} out of bounds, first {bad[0].tolist()}: {err[tuple(bad[0])]:.3e} > "
                           f"{bound[tuple(bad[0])]:.3e}")


def mass(c, cache, layer, q, q_lens, lens, RK, scale, lse, before):
    """attn_mass over a copy of `before` [B][Hkv][cap]: (mass, bound).  A score: rotation of q (2 D roundings), two fp16 parts
    (2^-22), codes' products cut off 2^-20 below the largest (their fp16 fields), so 2^-18 in all of sum |q'| times the
    largest level's distance from zero, 3 max |k'|; exp 2^-22; rows added up in float32."""
    B, n, Hq, D = q.shape
    Rk = np.asarray(O.rotations_of(c, RK, RK)[0], np.float64)
    out = np.array(before, np.float64)
    bound = np.full(out.shape, 1e-30)
    for b in range(B):
        T = max(0, min(int(lens[b]), c.capacity))
        m = max(0, min(int(q_lens[b]), n))
        for h in range(c.num_kv_heads if T else 0):
            K = rows64(c, cache, layer, 0, b, h, T)
            err = np.abs(out[b, h, :T]) * F32
            for t in range(m):
                for i in range(h * c.G, h * c.G + c.G):
                    ref = float(lse[b, t, i])
                    last = T - m + t
                    if not math.isfinite(ref) or last < 0:
                        continue
                    qr = np.asarray(q[b, t, i], np.float64) @ Rk
                    p = np.where(np.arange(T) <= last, np.exp(K @ qr * scale - ref), 0)
                    ds = scale * np.abs(qr).sum() * 3 * np.abs(K).max() * ((2 * D + 16) * F32 + 2.0 ** -18) / math.sqrt(D) * 2
                    out[b, h, :T] += p
                    err += p * (2 * ds + 2.0 ** -21 + 8 * F32 * abs(ref))
            bound[b, h, :T] += err + (m * c.G + 4) * F32 * np.abs(out[b, h, :T])
    return out, bound


def evict_choice(mass, T, S, W, keep):
    """Positions between sink and window that one (sequence, KV head) keeps, and its new length."""
    body = max(0, T - W - S) if T > S else 0
    x = np.where(np.isnan(mass[S:S + body]), -np.inf, mass[S:S + body])
    # a NaN is below -inf: by value, then by kind, then by position
    order = sorted(range(body), key=lambda i: (-x[i], bool(np.isnan(mass[S + i])), i))
    kept = sorted(order[:keep])
    return [S + i for i in kept], T - body + len(kept)
