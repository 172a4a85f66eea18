"""Definitions in 64 bits of the 8-bit cache and of attention over it, for the
tests (numpy; written apart from the kernels and from the timed plain forms)."""
import numpy as np

BASE = 10000.0


def e4m3_values():
    """The value of every code 0 .. 255 (NaN for 127 and 255)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


VALUES = e4m3_values()


def quantise(x):
    """(codes, scale bytes) of rows x [..., 64]: per row the smallest power of
    two that holds it, per value the nearest e4m3 value, ties to the even code."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    top = np.where(fin, np.abs(x), 0).max(-1)
    byte = np.zeros(top.shape, np.int64)
    for s in range(-127, 128):  # the first that holds it stays
        byte = np.where(top > 448 * 2.0 ** s, s + 128, byte)
    y = np.where(fin, x, 0) / 2.0 ** (byte[..., None] - 127.0)
    mag = VALUES[:127]  # ascending
    i = np.clip(np.searchsorted(mag, np.abs(y)), 1, 126)
    lo, hi = np.abs(y) - mag[i - 1], mag[i] - np.abs(y)
    code = np.where(lo < hi, i - 1, np.where(hi < lo, i, np.where(i % 2 == 0, i, i - 1)))
    code = np.where(np.signbit(x), code + 128, code)
    code = np.where(fin, code, 127)
    return code.astype(np.uint8), byte.astype(np.uint8)


def held(codes, scale):
    """What the rows stand for."""
    return VALUES[codes] * 2.0 ** (scale.astype(np.float64) - 127)[..., None]


def turn(x, pos, base=BASE):
    """x [n, heads, 64] rotated at pos [n]."""
    a = np.asarray(pos, np.float64)[:, None] * np.float64(np.float32(base)) ** (-2.0 * np.arange(32) / 64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    x1, x2 = x[..., :32], x[..., 32:]
    return np.concatenate([x1 * c - x2 * s, x1 * s + x2 * c], -1)


def decode(q, q_pos, K, V, pos, dtype):
    """One request: q [Hq, 64] raw, K, V [n, Hkv, 64] as held.  (out, tolerance).

    Tolerance.  The kernel's rotated key component is off by at most
    c (|x1| + |x2|): bf16, an fp16 rotation: three roundings of 2^-11 (the
    coefficient, one product, the sum); fp32: angles good to 4e-7 < 2^-21, three
    roundings of 2^-24, doubled: 2^-20.  The rotated query: its angles', 2^-20 (bf16
    as well: two fp16 parts).  So a score is off by at most
      E = sum_d (c + 2^-20) |q_d| (|x1| + |x2|)_d / 8 + 2^-18 sum_d |q_d k_d| / 8,
    with |q_d| bounded by its pair's sum, and a weight by 2 E relative to the
    normalised sum.  bf16 also rounds each weight to fp16: 2^-11 of it, or, for
    a small one, 2^-25 where the largest weighted value scale of its split
    counts at least 2^7 and a code 448 at most: 2^-23 of it."""
    Hq, n = q.shape[0], K.shape[0]
    if n == 0:
        return np.zeros((Hq, 64)), np.zeros((Hq, 64))
    G = Hq // K.shape[1]
    qr = turn(q[None], [q_pos])[0]
    Kr = np.repeat(turn(K, pos), G, axis=1)
    Vr = np.repeat(V, G, axis=1)
    pair = lambda x: np.abs(x) + np.abs(np.roll(x, 32, -1))  # noqa: E731
    s = np.einsum("hd,jhd->hj", qr, Kr) / 8
    c = 3 * 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20
    size = np.einsum("hd,jhd->hj", pair(q), np.repeat(pair(K), G, axis=1)) / 8
    E = ((c + 2.0 ** -20 + 2.0 ** -18) * size).max(-1)
    p = np.exp(s - s.max(-1, keepdims=True))
    tot = p.sum(-1, keepdims=True)
    w = p / tot
    out = np.einsum("hj,jhd->hd", w, Vr)
    A = np.einsum("hj,jhd->hd", w, np.abs(Vr))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = u * np.abs(out) + (np.expm1(2 * E)[:, None] + 2.0 ** -18) * A
    if dtype == "bf16":
        big = (w * np.abs(Vr).max(-1).T).max(-1)  # at most 448 scales, at least 224
        tol += 2.0 ** -11 * A + n * 2.0 ** -23 * big[:, None] / 224
    return out, tol


def attend(q, parts, dtype):
    """Rows q [m, Hq, 64] (rotated) over parts [(K, V [n, Hkv, 64], seen [m])]:
    (out, lse, tolerances), as the chunk calls' tests derive them."""
    m, Hq, _ = q.shape
    ss, sizes, vs = [], [], []
    for K, V, seen in parts:
        G = Hq // K.shape[1]
        Kr = np.repeat(K, G, axis=1)
        s = np.einsum("ihd,jhd->ihj", q, Kr) / 8
        size = np.einsum("ihd,jhd->ihj", np.abs(q), np.abs(Kr)) / 8
        hid = (np.arange(K.shape[0])[None] >= np.asarray(seen)[:, None])[:, None]
        ss.append(np.where(hid, -np.inf, s))
        sizes.append(np.where(hid, 0, size))
        vs.append(np.repeat(V, G, axis=1))
    s, size, V = np.concatenate(ss, -1), np.concatenate(sizes, -1), np.concatenate(vs, 0)
    E = 2.0 ** -18 * size.max(-1, initial=0)
    none = np.isneginf(s).all(-1)
    top = np.where(none, 0, s.max(-1, initial=-np.inf))
    p = np.where(np.isneginf(s), 0, np.exp(s - top[..., None]))
    tot = np.where(none, 1, p.sum(-1))
    p /= tot[..., None]
    # a hidden value that is not finite has no part
    V = np.where(np.isfinite(V), V, 0)
    out = np.einsum("ihj,jhd->ihd", p, V)
    A = np.einsum("ihj,jhd->ihd", p, np.abs(V))
    lse = np.where(none, -np.inf, top + np.log(tot))
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = u * np.abs(out) + (u + 2 * E[..., None] + 2.0 ** -18) * A
    return out, lse, tol, E + 2.0 ** -21 * (1 + np.abs(np.where(none, 0, lse)))
