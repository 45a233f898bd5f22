"""64-bit numpy references of the block-scaled FP8 experts and of the balance
loss, and the error bounds their tests use.  Independent of the library."""
import numpy as np

BLK = 128
U24 = 2.0 ** -24  # half a step of fp32, relative
U8 = 2.0 ** -8    # half a step of bf16
U4 = 2.0 ** -4    # half a step of E4M3


def decode_table():
    """Value of each E4M3 code (NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    sign, e, m = np.where(c & 0x80, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v[(c & 0x7F) == 0x7F] = np.nan
    return sign * v


TABLE = decode_table()
POS = TABLE[:127]  # 0 .. 448, ascending


def decode(codes):
    return TABLE[np.asarray(codes, np.uint8)]


def encode(v):
    """Nearest E4M3 code, ties to the even code; |v| <= 448."""
    a = np.abs(np.asarray(v, np.float64))
    hi = np.clip(np.searchsorted(POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - POS[lo], POS[hi] - a
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def exponent(amax):
    """Smallest e >= -127 with amax <= 448 * 2^e; 0 for amax 0."""
    amax = np.asarray(amax, np.float64)
    m, x = np.frexp(amax)
    return np.where(amax > 0, np.maximum(np.where(m <= 0.875, x - 9, x - 8), -127), 0)


def quantise(v, block_rows=1):
    """codes [R][K] and scale exponents [ceil(R / block_rows)][K / 128] of float64 v."""
    R, K = v.shape
    pad = np.zeros((-R % block_rows, K))
    b = np.concatenate([v, pad]).reshape(-1, block_rows, K // BLK, BLK)
    e = exponent(np.abs(b).max(axis=(1, 3)))
    q = encode(np.ldexp(b, -e[:, None, :, None])).reshape(-1, K)[:R]
    return q, e


def widen_rows(codes, e):
    return (decode(codes).reshape(codes.shape[0], -1, BLK) * np.exp2(e.astype(np.float64))[:, :, None]).reshape(
        codes.shape)


def widen_matrix(codes, s):
    """[n][K] codes with scales s [n/128][K/128] (numbers)."""
    return decode(codes) * np.repeat(np.repeat(np.asarray(s, np.float64), BLK, 0), BLK, 1)


def product(a, w):
    """a w^T in 64 bits, and a bound on what the FP8 matrix cores make of it.
    The products of E4M3 codes (4 x 4 bits) are exact.  The cores add those of
    neighbouring values on a grid of 2^-13 of the group's largest (measured for
    gfx950): each group's sum is off by at most 2^-13 max |a w| <= 2^-13 times the
    group's sum of |a w|, so all groups together by 2^-13 sum |a||w|.  The groups'
    sums then take at most K fp32 additions and the scales' products, K + 8
    roundings of at most U24 of the sum of magnitudes each.  (One product left
    out of K <= 2304 even ones is 2^-11.2 of that sum.)"""
    K = a.shape[1]
    return a @ w.T, (2.0 ** -13 + (K + 8) * U24) * (np.abs(a) @ np.abs(w).T)


def hidden(a, w, act, F):
    """h = act(a w^T) in 64 bits and a bound on the fp32 result.  SwiGLU:
    |silu'| <= 1.1; exp(-u) from an exponent rounded to fp32 (relative error of
    the exponential at most 4 U24 (1 + 2|u|)), a division and two products."""
    u, du = product(a, w)
    if act == "relu":
        return np.maximum(u, 0.0), du
    g, v, dg, dv = u[:, :F], u[:, F:], du[:, :F], du[:, F:]
    sg = 0.5 * (1.0 + np.tanh(0.5 * g))
    h = g * sg * v
    return h, (1.1 * dg + 16 * U24 * (1 + 2 * np.abs(g)) * np.abs(g * sg)) * (np.abs(v) + dv) + np.abs(g * sg) * dv


def check_quantised(codes, e, h, dh, what):
    """codes and scale exponents against h known to within dh: the scale is the
    least one for a value of that range, and every code within half a step."""
    s = np.exp2(e.astype(np.float64))
    hb, db = (v.reshape(v.shape[0], -1, BLK) for v in (h, dh))
    top, slack = np.abs(hb).max(axis=2), db.max(axis=2)
    assert np.all(top - slack <= 448 * s), f"{what}: a scale too small"
    low = (top + slack > 224 * s) | (e == -127) | ((top <= slack) & (e == 0))
    assert np.all(low), f"{what}: a scale too large"
    got = widen_rows(codes, e).reshape(hb.shape)
    bound = db + np.maximum(U4 * (np.abs(hb) + db), 2.0 ** -10 * s[:, :, None])
    over = np.abs(got - hb) - bound
    assert np.all(over <= 0), f"{what}: {over.max():.3e} beyond half a step"


def code_slack(h, dh):
    """Quantised h in 64 bits, and how far a quantisation of a value within dh
    of h may lie from it."""
    R, F = h.shape
    q, e = quantise(h)
    v = widen_rows(q, e)
    hb, db = h.reshape(R, -1, BLK), dh.reshape(R, -1, BLK)
    s = np.exp2(e.astype(np.float64))[:, :, None]
    near = [np.clip((hb + sign * db) / s, -448, 448) for sign in (-1, 1)]
    away = np.maximum(*[np.abs(decode(encode(n)) * s - v.reshape(hb.shape)) for n in near])
    top, slack = np.abs(hb).max(axis=2), db.max(axis=2)
    # a block whose largest value may lie on either side of a scale's border:
    # either grid rounds to within half a step of the coarser one
    border = exponent(np.maximum(top - slack, 0)) != exponent(top + slack)
    loose = db + 4 * np.maximum(U4 * (np.abs(hb) + db), 2.0 ** -10 * s)
    away = np.where(border[:, :, None], np.maximum(away, loose), away)
    return v, away.reshape(R, F)


# ---------------------------------------------------------------- balance loss
def balance(z, idx, offsets, aux_coef, z_coef, normalize=False, lam=1.0):
    """counts, (aux, Z), dlogits (NaN rows outside every sequence) and the bound
    factor eps of each token's gradient; all in 64 bits."""
    z = z.astype(np.float64)
    T, E = z.shape
    k = idx.shape[1]
    S = len(offsets) - 1
    counts = np.zeros((S, E), np.int64)
    dz, bound = np.full((T, E), np.nan), np.zeros((T, E))
    n = np.diff(offsets)
    some, total = max(1, int((n > 0).sum())), max(1, int(n.sum()))
    aux = zl = 0.0
    for s in range(S):
        if n[s] == 0:
            continue
        r = slice(offsets[s], offsets[s + 1])
        ids = idx[r].reshape(-1)
        np.add.at(counts[s], ids[(ids >= 0) & (ids < E)], 1)
        f = counts[s] / (n[s] * k)
        zt = z[r]
        top = zt.max(axis=1, keepdims=True)
        live = np.isfinite(top)
        with np.errstate(invalid="ignore"):
            q = np.where(live, np.exp(zt - np.where(live, top, 0)), 0.0)
        tot = q.sum(axis=1, keepdims=True)
        lse = np.where(live, np.where(live, top, 0) + np.log(np.where(live, tot, 1)), 0.0)
        q = q / np.where(live, tot, 1)
        spread = np.where(np.isfinite(zt), np.where(live, top, 0) - np.where(np.isfinite(zt), zt, 0), 0.0).max(
            axis=1, keepdims=True)
        if normalize:
            mu, sd = zt.mean(axis=1, keepdims=True), zt.std(axis=1, keepdims=True)
            zh = np.where(sd > 0, (zt - mu) / np.where(sd > 0, sd, 1), 0.0)
            p = np.exp(lam * (zh - zh.max(axis=1, keepdims=True)))
            p /= p.sum(axis=1, keepdims=True)
            spread = np.maximum(spread, lam * (zh.max(axis=1, keepdims=True) - zh.min(axis=1, keepdims=True)))
        else:
            p = q
        inner = p @ f
        aux += E * inner.sum() / n[s] / some
        zl += (lse ** 2).sum() / total
        ds = p * (f - inner[:, None])
        mag = p * (f + inner[:, None])
        if normalize:
            r1 = np.where(sd > 0, lam / np.where(sd > 0, sd, 1), 0.0)
            ds = r1 * (ds - ds.mean(axis=1, keepdims=True) - zh * (ds * zh).mean(axis=1, keepdims=True))
            mag = r1 * (mag + mag.mean(axis=1, keepdims=True) + np.abs(zh) * (mag * np.abs(zh)).mean(axis=1, keepdims=True))
        ca, cz = aux_coef * E / (some * n[s]), 2 * z_coef / total
        dz[r] = ca * ds + cz * lse * q
        # exp of a difference rounded to fp32: relative spread * U24; expf, the
        # sums over E (a tree and at most 16 in a row) and the products: 64 U24
        eps = (spread + 64) * U24
        # lse carries an absolute error of U24 |top| too
        bound[r] = 4 * eps * (abs(ca) * mag + abs(cz) * (np.abs(lse) + 1) * q) + 1e-40
    return counts, np.array([aux, zl]), dz, bound
