"""64-bit numpy references of the MXFP4 experts and of the orthogonalised update,
and the error bounds their tests use.  Independent of the library."""
import numpy as np

BLK = 32
U24 = 2.0 ** -24  # half a step of fp32, relative
U11 = 2.0 ** -11  # half a step of fp16
U8 = 2.0 ** -8    # half a step of bf16
POS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = np.concatenate([POS, -POS])


def encode(v):
    """Nearest E2M1 code, ties to the even code; |v| <= 6."""
    a = np.abs(np.asarray(v, np.float64))
    hi = np.clip(np.searchsorted(POS, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - POS[lo], POS[hi] - a
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def exponent(amax):
    """Smallest e >= -127 with amax <= 6 * 2^e; 0 for amax 0."""
    amax = np.asarray(amax, np.float64)
    m, x = np.frexp(amax)
    return np.where(amax > 0, np.maximum(np.where(m <= 0.75, x - 3, x - 2), -127), 0)


def pack(c):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    return np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)


def quantise(v):
    """Packed codes [..., K/2] and scale exponents [..., K/32] of finite float64 v [..., K]."""
    b = v.reshape(*v.shape[:-1], -1, BLK)
    e = exponent(np.abs(b).max(axis=-1))
    return pack(encode(np.ldexp(b, -e[..., None])).reshape(v.shape)), e


def widen(codes, e):
    """The values of packed codes with scale exponents e."""
    v = TABLE[unpack(codes)]
    b = v.reshape(*v.shape[:-1], -1, BLK)
    return (b * np.exp2(np.asarray(e, np.float64))[..., None]).reshape(v.shape)


def product(a, w):
    """a w^T in 64 bits, and a bound on what the matrix cores make of it.  The
    products of E2M1 codes are exact; the cores add those of neighbouring values on
    a grid of 2^-13 of the group's largest (measured for gfx950's f8f6f4 products),
    off by at most 2^-13 of each group's sum of |a w|; the groups' sums take at most
    K fp32 additions of at most U24 of the sum of magnitudes each."""
    K = a.shape[1]
    return a @ w.T, (2.0 ** -13 + (K + 8) * U24) * (np.abs(a) @ np.abs(w).T)


def hidden(a, w, act, F):
    """h = act(a w^T) in 64 bits and a bound on the fp32 result.  SwiGLU: |silu'| <=
    1.1; exp(-u) from an exponent rounded to fp32 (relative error of the exponential
    at most 4 U24 (1 + 2|u|)), a division and two products."""
    u, du = product(a, w)
    if act == "relu":
        return np.maximum(u, 0.0), du
    g, v, dg, dv = u[:, :F], u[:, F:], du[:, :F], du[:, F:]
    sg = 0.5 * (1.0 + np.tanh(0.5 * g))
    h = g * sg * v
    return h, (1.1 * dg + 16 * U24 * (1 + 2 * np.abs(g)) * np.abs(g * sg)) * (np.abs(v) + dv) + np.abs(g * sg) * dv


def half_step(a, s):
    """Half the spacing of the codes around |v| = a (at most 6 s) under scale s: 1/4, 1/2
    or 1 of s, where a value next to a border of spacings counts to the wider one."""
    return np.where(a <= 2 * s, 0.25, np.where(a <= 4 * s, 0.5, 1.0)) * s


def check_quantised(codes, e, h, dh, what):
    """codes and scale exponents against h known to within dh: the scale is the
    least one for a value of that range, and every code within half a step."""
    s = np.exp2(e.astype(np.float64))
    hb, db = (v.reshape(v.shape[0], -1, BLK) for v in (h, dh))
    top, slack = np.abs(hb).max(axis=2), db.max(axis=2)
    assert np.all(top - slack <= 6 * s), f"{what}: a scale too small"
    low = (top + slack > 3 * s) | (e == -127) | ((top <= slack) & (e == 0))
    assert np.all(low), f"{what}: a scale too large"
    got = widen(codes, e).reshape(hb.shape)
    bound = db + half_step(np.abs(hb) + db, s[:, :, None])
    over = np.abs(got - hb) - bound
    assert np.all(over <= 1e-12 * s[:, :, None]), f"{what}: {over.max():.3e} beyond half a step"


def code_slack(h, dh):
    """Quantised h in 64 bits, and how far a quantisation of a value within dh
    of h may lie from it."""
    R, F = h.shape
    q, e = quantise(h)
    v = widen(q, e)
    hb, db = h.reshape(R, -1, BLK), dh.reshape(R, -1, BLK)
    s = np.exp2(e.astype(np.float64))[:, :, None]
    near = [np.clip((hb + sign * db) / s, -6, 6) for sign in (-1, 1)]
    away = np.maximum(*[np.abs(TABLE[encode(n)] * s - v.reshape(hb.shape)) for n in near])
    top, slack = np.abs(hb).max(axis=2), db.max(axis=2)
    # a block whose largest value may lie on either side of a scale's border: either
    # grid rounds to within half a step of the coarser one
    border = exponent(np.maximum(top - slack, 0)) != exponent(top + slack)
    loose = db + 4 * half_step(np.minimum(np.abs(hb) + db, 12 * s), s)
    away = np.where(border[:, :, None], np.maximum(away, loose), away)
    return v, away.reshape(R, F)


# ---------------------------------------------------------------- orthogonalised update
COEF = (3.4445, -4.7750, 2.0315)


def momentum(g, m, beta, nesterov):
    """(new momentum, update), in 64 bits."""
    if m is None:
        return None, g
    m = beta * m + g
    return m, g + beta * m if nesterov else m


def orthogonal(u, steps):
    """The Newton-Schulz iterate of one matrix, by its singular values: each goes
    through the quintic by itself, the singular vectors stay."""
    n = np.linalg.norm(u)
    if n == 0:
        return np.zeros_like(u)
    left, s, right = np.linalg.svd(u / n, full_matrices=False)
    a, b, c = COEF
    for _ in range(steps):
        s = s * (a + b * s ** 2 + c * s ** 4)
    return (left * s) @ right


def orthogonal_by_products(u, steps):
    """The same by the products of the definition."""
    x = u / np.linalg.norm(u)
    wide = u.shape[0] <= u.shape[1]
    a, b, c = COEF
    for _ in range(steps):
        s = x @ x.T if wide else x.T @ x
        p = a * np.eye(len(s)) + b * s + c * s @ s
        x = p @ x if wide else x @ p
    return x


def orthogonal_fp16(u, steps):
    """orthogonal() with the roundings that the fp16 products make, and no others: X,
    A and B as operands (scaled by powers of two), the diagonals of A and B and the
    first term a X exact, the diagonal's term on the fp16 X up to the last two steps."""
    x = u if u.shape[0] <= u.shape[1] else u.T
    x = x / np.linalg.norm(x) if np.any(x) else x
    sx, sa = 2.0 ** np.floor(np.log2(np.sqrt(x.shape[1]))), 2.0 ** 14
    a, b, c = COEF

    def half(v, s):
        return (v * s).astype(np.float16).astype(np.float64) / s

    for i in range(steps):
        xh = half(x, sx)
        full = xh @ xh.T
        d = np.diag(full).copy()
        o = half(full - np.diag(d), sa)
        p = c * (o @ o + (d[:, None] + d[None, :]) * o) + b * o
        db = np.diag(p) + b * d + c * d * d
        p = half(p - np.diag(np.diag(p)), sa)
        x = a * x + db[:, None] * (x if i >= steps - 2 else xh) + p @ xh
    return x
