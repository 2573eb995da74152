"""Plain 64-bit (numpy) forms of the 8-bit operators, and error bounds.

Nothing here is shared with the library: e4m3 rounding works on exponents from
frexp, bytes are decoded from their bit fields."""
import numpy as np

MIN_AMAX = 448.0 * 2.0 ** -64


def e4m3_round(y):
    """Nearest e4m3 value, ties to even, saturating (y: float64)."""
    y = np.asarray(y, np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(y), y, 0.0))
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        r = np.clip(np.rint(np.where(np.isfinite(y), y, 0.0) / step) * step, -448.0, 448.0)
        r = np.where(np.isinf(y), np.sign(y) * 448.0, r)
    return np.where(np.isnan(y), np.nan, r)


def e4m3_decode(b):
    """Values of e4m3 bytes from their bit fields."""
    b = np.asarray(b, np.uint8).astype(np.int64)
    s, e, m = b >> 7, (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


def quant(x, block_rows):
    """(values, scale): x float64 [rows][cols]; fp32 roundings made in order."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    q = np.empty_like(x)
    s = np.empty((-(-rows // block_rows), -(-cols // 128)), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            sl = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            p = x[sl]
            f = np.abs(p[np.isfinite(p)])
            a = np.float32(max(f.max() if f.size else 0.0, MIN_AMAX))
            s[i, j] = a / np.float32(448.0)
            inv = np.float32(448.0) / a
            with np.errstate(invalid="ignore", over="ignore"):
                q[sl] = e4m3_round(p.astype(np.float32) * inv)
    return q, s


def matmul(xq, xs, wq, ws):
    """(Y, envelope): the envelope sums the terms' magnitudes."""
    k = xq.shape[1]
    sx = np.repeat(xs.astype(np.float64), 128, 1)[:, :k]
    sw = np.repeat(np.repeat(ws.astype(np.float64), 128, 0)[:wq.shape[0]], 128, 1)[:, :k]
    a, b = xq * sx, wq * sw
    return a @ b.T, np.abs(a) @ np.abs(b).T


def matmul_bound(env, k):
    """fp32 accumulation of exact products: a block's sum of 128, then one scaled
    addition per block.  Each addition errs by at most one unit in the last place
    (2^-23, also for an accumulator that truncates) of a partial sum that is at
    most env; the product of the scales and its product with the sum round twice
    more by 2^-24."""
    return (min(k, 128) + -(-k // 128) + 2) * 2.0 ** -23 * env


def append(cache, new, table, lens, off, i8):
    """Append to float64 stored values cache["k"], ["v"] [pages][H][P][D] and
    scales cache["k_scale"], ["v_scale"], in place; new = {"k", "v"} [rows][H][D]."""
    H, P = cache["k"].shape[1], cache["k"].shape[2]
    most = 127.0 if i8 else 448.0

    def to8(y):
        return np.clip(np.rint(y), -127, 127) if i8 else e4m3_round(y)

    for b, t in enumerate(lens):
        n = off[b + 1] - off[b]
        if t == 0 or n == 0:
            continue
        start = t - n
        for slot in range(start // P, -(-t // P)):
            page, lo, hi = table[b][slot], max(start, slot * P), min(t, slot * P + P)
            for w in "kv":
                x = new[w][off[b] + lo - start:off[b] + hi - start].astype(np.float64)
                for h in range(H):
                    y = x[:, h]
                    f = np.abs(y[np.isfinite(y)])
                    e, big = -40, f.max() if f.size else 0.0
                    while e < 60 and most * 2.0 ** e < big:
                        e += 1
                    scale, old = np.float32(2.0 ** e), lo - slot * P
                    if old:
                        had = cache[w + "_scale"][page, h]
                        scale = max(scale, had)
                        if scale != had:
                            cache[w][page, h, :old] = to8(cache[w][page, h, :old] * (np.float64(had) / scale))
                    with np.errstate(invalid="ignore"):
                        z = to8(np.where(np.isnan(y), 0.0, y) / scale)
                    cache[w][page, h, old:hi - slot * P] = z
                    cache[w + "_scale"][page, h] = scale


def attention(cache, q, table, lens, off, scale, window=0, sinks=0):
    """(O, lse, bound of O, bound of lse), float64; q [rows][heads][D].

    Bounds: S errs by the fp32 accumulation of D exact products and by three
    more roundings (scales), each at most 2^-23 of the sum of magnitudes; adding
    log2 of the value scale and subtracting the maximum round twice at the size
    of |S| + 64; exp2 errs by 2^-22 relative.  A probability is then rounded to
    11 bits: 2^-11 relative, or half of fp16's smallest step, 2^-25, where the
    largest one is held as at least 2^4; that is 2^-29 of the largest product of
    a probability and its page's scale, and a page's largest value is at least
    half of its format's.  Numerator and
    denominator carry these errors, the output one rounding to bf16 (2^-8)."""
    P = cache["k"].shape[2]
    H = cache["k"].shape[1]
    rows, heads, D = q.shape
    G = heads // H
    O, lse = np.zeros((rows, heads, D)), np.full((rows, heads), -np.inf)
    bO, bl = np.zeros((rows, heads, D)), np.zeros((rows, heads))
    for b, t in enumerate(lens):
        n = off[b + 1] - off[b]
        if t == 0:
            continue
        ids = np.array(table[b][:-(-t // P)])
        K = (cache["k"][ids] * cache["k_scale"][ids].astype(np.float64)[:, :, None, None])
        V = (cache["v"][ids] * cache["v_scale"][ids].astype(np.float64)[:, :, None, None])
        K = K.transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :t]
        V = V.transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :t]
        tok = np.arange(t)
        for i in range(n):
            p = t - n + i
            see = tok <= p
            if window:
                see &= (tok > p - window) | (tok < sinks)
            if not see.any():
                continue
            for hd in range(heads):
                h = hd // G
                x = q[off[b] + i, hd].astype(np.float64)
                k, v = K[h][see], V[h][see]
                s = scale * (k @ x)
                env = np.abs(scale) * (np.abs(k) @ np.abs(x)).max()
                top = s.max()
                w = np.exp(s - top)
                den = w.sum()
                r = off[b] + i
                O[r, hd] = w @ v / den
                lse[r, hd] = top + np.log(den)
                es = (D + 6) * 2.0 ** -23 * env + 2 * 2.0 ** -24 * (env * 1.45 + 64) + 2.0 ** -22
                mag = w @ np.abs(v) / den
                small = see.sum() * 2.0 ** -28 * np.abs(v).max()
                bO[r, hd] = (2 * es + 2.0 ** -11 + 2.0 ** -20) * mag + 2.0 ** -8 * np.abs(O[r, hd]) + small
                bl[r, hd] = es + 2.0 ** -20 + 2.0 ** -22 * abs(lse[r, hd])
    return O, lse, bO, bl
