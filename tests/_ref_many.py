"""64-bit references of the many-row path (top-k gating, sorted picks, MXFP4 rows and
products), in numpy, written from the definitions in ``include/moeblk.h``, and the
tolerances that follow from them."""

import numpy as np

U24 = 2.0**-24
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def half_step(kind):
    return {"bf16": 2.0**-8, "fp32": U24}[kind]


# ------------------------------------------------------------------ MXFP4


def padded(K):
    return -(-K // 128) * 128


def mx_scale(amax):
    """e (an int array), the smallest >= -127 with amax < 7 2^e; 128 where amax is not finite."""
    e = np.full(amax.shape, -127)
    fin = np.isfinite(amax)
    for k in range(-127, 127):
        big = fin & (amax >= 7.0 * 2.0**k)
        if not big.any():
            break
        e[big] = k + 1
    e[~fin] = 128
    return e


def mx_codes(v):
    """Nearest e2m1 code (ties to the even one) of |v| < 7; the sign bit is v's."""
    a = np.abs(v)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")
    up = np.searchsorted(mid, a, side="right")
    code = np.where((lo != up) & (lo % 2 == 1), up, lo)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def mx_quant(x):
    """x [M, K] float64 -> codes [M, Kp] (one a byte), scale bytes [M, Kp / 32]."""
    M, K = x.shape
    v = np.zeros((M, padded(K)))
    v[:, :K] = x
    v = v.reshape(M, -1, 32)
    mag = np.abs(v)
    amax = np.where(np.isfinite(mag).all(axis=2), mag.max(axis=2), np.inf)
    e = mx_scale(amax)
    ok = (e < 128)[:, :, None]
    code = np.where(ok, mx_codes(np.where(ok, v, 0.0) / np.exp2(e.astype(np.float64))[:, :, None]), 0)
    return code.reshape(M, -1).astype(np.uint8), (e + 127).astype(np.uint8)


def mx_unpack(q):
    """[M, n] bytes -> [M, 2 n] codes, the low nibble first."""
    return np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], -1)


def mx_pack(code):
    return (code[..., ::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def mx_values(code, s):
    """float64 values of codes [..., K] and scale bytes [..., K / 32]; byte 255 is NaN."""
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    f = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127.0))
    return (v.reshape(*s.shape, 32) * f[..., None]).reshape(code.shape)


def product(x, w):
    """Rows [M, K] times a weight [N, K], and the sum of magnitudes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def product_tol(mag, K):
    """fp32 sums, each addition off by at most one unit in the last place of the running
    sum (which a truncating adder keeps to as well): 128 products an instruction, one
    instruction a chunk, then up to 8 waves and 32 K parts. The scales are exact."""
    return (128 + -(-K // 128) + 8 + 32) * 2.0**-23 * mag


def swiglu(g, u):
    return g / (1.0 + np.exp(-g)) * u


def swiglu_tol(g, u, tg, tu):
    """|silu'| <= 1.1; in fp32 the exponential's argument is off by |g| 2^-24, its result,
    the sum, the division and two products by a unit each."""
    s = g / (1.0 + np.exp(-g))
    h = s * u
    return 1.1 * tg * (np.abs(u) + tu) + np.abs(s) * tu + (np.abs(g) + 8) * 2 * U24 * np.abs(h)


# ------------------------------------------------------------------ gate


def gate(l, bias, topk, score, renorm):
    """ids, w of logits [T, E] (float32 values), bias [E] float32 or None."""
    T, E = l.shape
    key = l.astype(np.float32) if bias is None else (l.astype(np.float32) + bias.astype(np.float32)[None, :])
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        k = key[t].astype(np.float64)
        rank = np.where(np.isnan(k), np.inf, k)
        order = sorted((e for e in range(E) if not k[e] == -np.inf), key=lambda e: (not np.isnan(k[e]), -rank[e], e))
        pick = order[:topk]
        ids[t, :len(pick)] = pick
        w[t, :len(pick)] = pick_weights(l[t].astype(np.float64), pick, score, renorm)
    return ids, w


def _log_scores(row, score):
    if score == "sigmoid":
        return np.minimum(row, 0.0) - np.log1p(np.exp(-np.abs(row)))
    return row


def pick_weights(row, pick, score, renorm):
    """Weights of the picks (expert ids) of one row of logits."""
    pick = list(pick)
    if not pick:
        return np.zeros(0)
    a = _log_scores(row, score)
    if score == "sigmoid" and not renorm:
        return np.exp(a[pick])
    over = a[pick] if renorm else a
    m = np.max(over)
    if m == -np.inf:
        return np.zeros(len(pick))
    return np.exp(a[pick] - m) / np.exp(over - m).sum()


def gate_grad(l, ids, g, score, renorm):
    """dlogits [T, E] and, per value, the sum of the magnitudes of its terms."""
    T, E = l.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        row = l[t].astype(np.float64)
        slots = [s for s in range(ids.shape[1]) if 0 <= ids[t, s] < E]
        pick = [int(ids[t, s]) for s in slots]
        w = pick_weights(row, pick, score, renorm)
        gs = np.array([g[t, s] for s in slots], np.float64)
        mean, mmag = float(gs @ w), float(np.abs(gs) @ w)
        if score == "softmax" and not renorm:
            if not np.all(row == -np.inf):
                p = np.exp(row - row.max())
                p /= p.sum()
                out[t] -= mean * p
                mag[t] += mmag * p
            for e, wv, gv in zip(pick, w, gs):
                out[t, e] += wv * gv
                mag[t, e] += wv * abs(gv)
            continue
        for e, wv, gv in zip(pick, w, gs):
            slope = 1.0 / (1.0 + np.exp(min(row[e], 700.0))) if score == "sigmoid" else 1.0
            out[t, e] += wv * slope * (gv - (mean if renorm else 0.0))
            mag[t, e] += wv * slope * (abs(gv) + (mmag if renorm else 0.0))
    return out, mag


def gate_rel(l):
    """Relative error of a weight: the exponential's argument is a difference of logits,
    rounded once (|l - m| 2^-24 of the result); the exponentials, sums of up to 256 of
    them (16 in a lane, 4 steps across), reciprocal, division and products add at most
    40 units in the last place. Differences above 104 leave less than 2^-149."""
    fin = np.where(np.isfinite(l), l.astype(np.float64), 0.0)
    return (40 + np.minimum(2 * np.abs(fin).max(axis=1, keepdims=True), 104)) * 2 * U24


# ------------------------------------------------------------------ sorted picks


def sort_picks(ids, base, n):
    """counts, offsets, rows, pick_pos."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    lists = [np.nonzero(flat == base + e)[0] for e in range(n)]
    counts = np.array([len(p) for p in lists], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    order = np.concatenate(lists).astype(np.int64)
    rows = np.full(T * k, -1, np.int32)
    rows[:len(order)] = order // k
    pos = np.full(T * k, -1, np.int32)
    pos[order] = np.arange(len(order))
    return counts, offsets, rows, pos.reshape(T, k)


def weighted_sum(y, w, pos):
    """out [T, d] and the sums of magnitudes; w may be None."""
    T, k = pos.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for s in range(k):
        on = pos[:, s] >= 0
        f = np.ones(T) if w is None else w[:, s].astype(np.float64)
        v = f[on, None] * y[pos[on, s]]
        out[on] += v
        mag[on] += np.abs(v)
    return out, mag
