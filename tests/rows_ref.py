"""Plain 64-bit forms of kv_read, attn_extend and attn_decode_prefix over the
oracle's cached rows, and how far float32 / fp16 arithmetic may be from them."""
import math

import numpy as np

from oracle import oscar_oracle as O


def rows64(c, cache, layer, role, b, h, T):
    """Rotated rows [T][D] of one (sequence, KV head), as attention sees them."""
    return O.dequant_history(c, cache, layer, role, b, h, T)


def read(c, cache, layer, start, lens, n, RK, RV, k0, v0):
    """kv_read over copies of the buffers k0, v0."""
    rots = O.rotations_of(c, RK, RV)
    out = [np.array(k0, np.float64), np.array(v0, np.float64)]
    for b in range(c.batch):
        for role in (0, 1):
            R = np.asarray(rots[role], np.float64)
            if role and c.flags & O.FLAG_ABSORB_V:
                R = np.eye(c.head_dim)
            for h in range(c.num_kv_heads):
                T = min(int(lens[b]), c.capacity)
                if T < 1:
                    continue
                x = rows64(c, cache, layer, role, b, h, T) @ R.T
                for t in range(n):
                    p = int(start[b]) + t
                    if 0 <= p < T:
                        out[role][b, t, h] = x[p]
    return out


def score_error(q, K, scale, coarse):
    """Bound on the error of any score q . K[t] * scale.  In float32: D products
    and sums, each off by 2^-24 of the sum of magnitudes, twice that for the
    rotation of q, the scale and the exponent.  `coarse`: the tensor-core form
    s (4 sum_d q_d y_d) + (z - 4 s) sum_d q_d with y = 1 + code / 4, whose terms
    are at most 4 s 1.75 + |z| + 4 s <= 9 max_d |k_d| (s <= 2/3 max) times sum |q|."""
    size = (np.abs(K).max(1) * np.abs(q).sum() * 9 if coarse else np.abs(K) @ np.abs(q)).max()
    return 2 * (len(q) + 8) * 2.0 ** -24 * scale * size


def attend(q, K, V, hidden, scale, coarse):
    """One query row against rotated rows K, V [T][D]: (o', lse, bound on the
    2-norm of the error of o', bound on the error of lse).  A score error d
    changes probabilities by a factor within 1 +- 2 d; `coarse` adds the fp16
    rounding of probabilities and value rows (2^-11 each, and 2^-25 of the
    largest where they are subnormal); sums of T terms are float32."""
    T = len(K)
    see = ~hidden
    if not see.any():
        return np.zeros(K.shape[1]), -math.inf, 0.0, 0.0
    s = (K @ q) * scale
    s[hidden] = -math.inf
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    ds = score_error(q, K[see], scale, coarse)
    rel = 2 * ds + (T + 64) * 2.0 ** -24
    if coarse:
        rel += 2 * 2.0 ** -11 + T * 2.0 ** -24
    return ((p[see] @ V[see]) / l, m + math.log(l), rel * np.linalg.norm(V[see], axis=1).max(),
            ds + (T + 64) * 2.0 ** -24)


def finish(c, o, bound, RV, fp32):
    """Un-rotation and the output's rounding: (out, bound on the 2-norm of its error)."""
    R = np.asarray(O.rotations_of(c, None, RV)[1], np.float64)
    out = o if c.flags & O.FLAG_ABSORB_V else o @ R.T
    size = np.linalg.norm(o)
    return out, bound + (c.head_dim * 2.0 ** -24 * 2 + (0 if fp32 else 2.0 ** -8)) * size + 1e-30


def check_rows(name, got, want, bounds):
    """Every output row within its own bound."""
    err = np.linalg.norm(got - want, axis=-1)
    assert np.isfinite(err).all(), f"{name}: not finite at {np.argwhere(~np.isfinite(err))[:4].tolist()}"
    bad = np.argwhere(err > bounds)
    assert bad.size == 0, (f"{name}: {len(bad)} rows out of bounds, first {bad[0].tolist()}: "
                           f"{err[tuple(bad[0])]:.3e} > {bounds[tuple(bad[0])]:.3e}")


def check_lse(got, want, bounds):
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), "empty rows differ"
    ok = np.isfinite(want)
    err = np.abs(got[ok] - want[ok])
    lim = bounds[ok] + 4 * 2.0 ** -24 * np.abs(want[ok])
    assert (err <= lim).all(), f"lse: {err.max():.3e}, bound {lim[err.argmax()]:.3e}"


def extend(c, cache, layer, q, q_lens, lens, RK, RV, scale, out0, lse0, fp32):
    """attn_extend over copies of the buffers out0, lse0: (out, lse, out bounds, lse bounds)."""
    B, n, Hq, D = q.shape
    Rk = np.asarray(O.rotations_of(c, RK, RV)[0], np.float64)
    out, lse = np.array(out0, np.float64), np.array(lse0, np.float64)
    ob, lb = np.full((B, n, Hq), 1e-30), np.full((B, n, Hq), 1e-30)
    for b in range(B):
        T = max(0, min(int(lens[b]), c.capacity))
        m = min(int(q_lens[b]), n)
        for h in range(Hq):
            if m < 1:
                continue
            K = rows64(c, cache, layer, 0, b, h // c.G, T) if T else np.zeros((0, D))
            V = rows64(c, cache, layer, 1, b, h // c.G, T) if T else np.zeros((0, D))
            for t in range(m):
                hidden = np.arange(T) > T - m + t
                qr = np.asarray(q[b, t, h], np.float64) @ Rk
                o, lse[b, t, h], err, lb[b, t, h] = attend(qr, K, V, hidden, scale, not fp32)
                out[b, t, h], ob[b, t, h] = finish(c, o, err, RV, fp32)
    return out, lse, ob, lb


def prefix(c, cache, pc, pcache, layer, q, lens, plen, RK, RV, scale, fp32):
    """attn_decode_prefix: (out, lse, out bounds, lse bounds)."""
    B, Hq, D = q.shape
    Rk = np.asarray(O.rotations_of(c, RK, RV)[0], np.float64)
    out, lse = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    ob, lb = np.zeros((B, Hq)), np.zeros((B, Hq))
    P = min(int(plen), pc.capacity)
    for h in range(Hq):
        pk = rows64(pc, pcache, layer, 0, 0, h // c.G, P) if P else np.zeros((0, D))
        pv = rows64(pc, pcache, layer, 1, 0, h // c.G, P) if P else np.zeros((0, D))
        for b in range(B):
            T = max(0, min(int(lens[b]), c.capacity))
            K = np.concatenate([pk, rows64(c, cache, layer, 0, b, h // c.G, T) if T else np.zeros((0, D))])
            V = np.concatenate([pv, rows64(c, cache, layer, 1, b, h // c.G, T) if T else np.zeros((0, D))])
            qr = np.asarray(q[b, h], np.float64) @ Rk
            hidden = np.zeros(len(K), bool)
            o, lse[b, h], err, lb[b, h] = attend(qr, K, V, np.zeros(len(K), bool), scale, not fp32)
            out[b, h], ob[b, h] = finish(c, o, err, RV, fp32)
    return out, lse, ob, lb
