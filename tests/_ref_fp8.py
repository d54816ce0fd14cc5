"""64-bit references of the FP8 (block-128) products and the router's balance
loss, in numpy, written from the definitions in ``include/moeblk.h``."""

import numpy as np

BLK = 128
U24 = 2.0**-24


def e4m3_table() -> np.ndarray:
    """The 256 values of OCP e4m3: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; exponent 0 is subnormal, S.1111.111 is NaN, no infinities."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0**-9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


TABLE = e4m3_table()
_POS = TABLE[:127]
_MID = (_POS[1:] + _POS[:-1]) / 2


def e4m3_encode(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte (ties to the even mantissa) of |v| <= 448, NaN -> 0x7f."""
    a = np.abs(np.nan_to_num(v, nan=0.0))
    lo = np.searchsorted(_MID, a, side="left")  # a tie stays at the lower code
    up = np.searchsorted(_MID, a, side="right")
    code = np.where((lo != up) & (lo % 2 == 1), up, lo).astype(np.uint8)
    code = np.where(np.signbit(v), code | 0x80, code)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def block_scale(amax: np.ndarray) -> np.ndarray:
    """2^e, the smallest integer e >= -126 with amax <= 448 2^e; NaN if amax is not finite."""
    out = np.full(amax.shape, 2.0**-126)
    fin = np.isfinite(amax)
    for e in range(-126, 121):
        big = fin & (amax > 448.0 * 2.0**e)
        if not big.any():
            break
        out[big] = 2.0 ** (e + 1)
    out[~fin] = np.nan
    return out


def quant(x: np.ndarray):
    """x [M, K] float64 -> e4m3 bytes [M, Kp], scales [Kb, M] (float64)."""
    M, K = x.shape
    kb = -(-K // BLK)
    v = np.zeros((M, kb * BLK))
    v[:, :K] = x
    v = v.reshape(M, kb, BLK)
    mag = np.abs(v)
    amax = np.where(np.isfinite(mag).all(axis=2), mag.max(axis=2, initial=0.0), np.inf)
    s = block_scale(amax)
    q = e4m3_encode(v / s[:, :, None])
    return q.reshape(M, kb * BLK), np.ascontiguousarray(s.T)


def values(q, s):
    """What quantised rows stand for: [M, Kp] float64."""
    M = q.shape[0]
    return (TABLE[q].reshape(M, -1, BLK) * s.T[:, :, None]).reshape(M, -1)


def weight(q, s):
    """float64 [N, K] of e4m3 bytes and 128 x 128 block scales."""
    N, K = q.shape
    big = np.repeat(np.repeat(np.asarray(s, np.float64), BLK, 0), BLK, 1)[:N, :K]
    return TABLE[q] * big


def product(xv, w):
    """Rows [M, Kp] times a weight [N, K], and the sum of magnitudes."""
    K = w.shape[1]
    x = xv[:, :K]
    return x @ w.T, np.abs(x) @ np.abs(w).T


def product_tol(mag, K):
    """fp32 accumulation: 128 products a block and one sum over the blocks
    (the additions of 8 wave sums included), each addition off by at most one
    unit in the last place of the running sum (2^-23 also covers a truncating
    adder), plus one rounding for each of the two scale products."""
    return (BLK + -(-K // BLK) + 8 + 2) * 2.0**-23 * mag


def half_step(kind):
    return {"bf16": 2.0**-8, "fp32": U24}[kind]


def ffn_row_tol(xv, w13, w2):
    """y of rows [n, d] (dequantised) and a per-value bound on |y - exact| before
    the rounding to bf16: gate_up's accumulation error moves h, which can move
    a value of h across a rounding border (or its block across a scale
    border); each such move is bounded by quantising both ends of h's interval
    with both ends' scales."""
    n, d = xv.shape
    I = w2.shape[1]  # noqa: E741
    gu, mag = product(xv, w13)
    tol = product_tol(mag, d) + U24 * np.abs(gu)
    g, u = gu[:, :I], gu[:, I:]
    tg, tu = tol[:, :I], tol[:, I:]
    silu = lambda z: z / (1.0 + np.exp(-z))  # noqa: E731
    h = silu(g) * u
    # |silu'| <= 1.1; 8 ulp for exp, division and products in fp32
    th = 1.1 * tg * (np.abs(u) + tu) + np.abs(silu(g)) * tu + 8 * U24 * np.abs(h)
    hq, hs = quant(h)
    ref = values(hq, hs)
    lo, hi = np.maximum(np.abs(h) - th, 0.0), np.abs(h) + th
    move = np.zeros_like(h)
    b = h.reshape(n, -1, BLK)
    for amax in (lo.reshape(b.shape).max(axis=2), hi.reshape(b.shape).max(axis=2)):
        s = np.repeat(block_scale(amax), BLK, axis=1)
        for end in (h - th, h + th):
            v = TABLE[e4m3_encode(np.clip(end / s, -448, 448))] * s
            move = np.maximum(move, np.abs(v - ref))
    y, mag2 = product(ref, w2)
    return y, product_tol(mag2 + move @ np.abs(w2).T, I) + move @ np.abs(w2).T


# ------------------------------------------------------------------ balance


def balance_scores(l, score):
    """p and dp's factor (1 - sigmoid, or 1) of rows of logits (float64)."""
    p = np.zeros_like(l)
    f = np.ones_like(l)
    for t in range(l.shape[0]):
        row = l[t]
        if np.all(row == -np.inf):
            continue
        m = row.max()
        if score == "sigmoid":
            m = min(m, 0.0)
            s = np.exp(np.minimum(row, 0.0) - m) / (1.0 + np.exp(-np.abs(row)))
            f[t] = 1.0 / (1.0 + np.exp(np.minimum(row, 700.0)))
        else:
            s = np.exp(row - m)
        p[t] = s / s.sum()
    return p, f


def balance(l, ids, starts, n_seq, score, coef, dloss=1.0):
    """counts, probs, loss, dlogits (NaN outside the sequences), float64."""
    T, E = l.shape
    k = ids.shape[1]
    counts = np.zeros((n_seq, E), np.int64)
    probs = np.zeros((n_seq, E))
    grad = np.full((T, E), np.nan)
    loss = 0.0
    for b in range(n_seq):
        a, z = int(starts[b]), int(starts[b + 1])
        n = z - a
        if n <= 0:
            continue
        pick = ids[a:z].reshape(-1)
        pick = pick[(pick >= 0) & (pick < E)]
        counts[b] = np.bincount(pick, minlength=E)
        p, f = balance_scores(l[a:z].astype(np.float64), score)
        probs[b] = p.mean(axis=0)
        loss += coef / n_seq * E / (k * n) * float(counts[b] @ probs[b])
        w = dloss * coef / n_seq * E / (k * n * n) * counts[b]
        grad[a:z] = p * f * (w[None, :] - (p @ w)[:, None])
    return counts, probs, loss, grad
