"""What the sharper tests of the 8-bit decode compare (numpy, 64 bits): a request's
output as a vector, against a bound that a lost or repeated tile of 32 entries, or the
loss of the query's second fp16 part, passes many times over."""
import numpy as np

from _kv8 import held, quantise, turn


SPREAD = 0.25  # of the queries


def _one_head(q, K, V, kept):
    s = K @ q / 8
    s = np.where(kept > 0, s, -np.inf)
    w = kept * np.exp(s - s.max(initial=-np.inf)) if kept.any() else np.zeros(len(K))
    return w / w.sum() if kept.any() else w


def decode_norm(q, q_pos, K, V, pos, kept=None, rotated=True, terms=0.0):
    """One request, bf16: (out [Hq, 64], bound on the norm of each head's error).
    kept: how often each entry counts (once each); terms: the score's error as a part
    of sum |q_d k_d| / 8.

    The bound.  The output's rounding is at most 2^-8 of the output's norm.  A rotated
    key component is off by at most 3 * 2^-11 (|x1| + |x2|) (three roundings; none where
    the position is 0), a weight by 2^-11 of itself.  These errors differ from one
    component and entry to the next, so the score of entry j is off by a sum of
    independent terms, of variance at most d_j^2 = sum_d (3 * 2^-11 |q_d| pair_d / 8)^2,
    and the output by sum_j w_j e_j (v_j - out) with e_j of variance d_j^2 + 2^-22: six
    standard deviations of it are allowed, and 2^-18 sum_j w_j |v_j| for the sums in
    fp32."""
    Hq, n = q.shape[0], K.shape[0]
    if n == 0:
        return np.zeros((Hq, 64)), np.zeros(Hq)
    kept = np.ones(n) if kept is None else kept
    G = Hq // K.shape[1]
    qr, Kr = turn(q[None], [q_pos])[0], turn(K, pos)
    out, bound = np.zeros((Hq, 64)), np.zeros(Hq)
    for h in range(Hq):
        k, v, x = Kr[:, h // G], V[:, h // G], K[:, h // G]
        w = _one_head(qr[h], k, v, kept)
        out[h] = w @ v
        var = np.full(n, 2.0 ** -22)
        if rotated:
            pair = np.abs(x) + np.abs(np.roll(x, 32, -1))
            var += (3 * 2.0 ** -11 / 8) ** 2 * (pair ** 2 @ qr[h] ** 2)
        var += (terms * (np.abs(k) @ np.abs(qr[h])) / 8) ** 2
        norm = np.linalg.norm
        bound[h] = (2.0 ** -8 * norm(out[h]) + 6 * np.sqrt(np.sum(w ** 2 * var * norm(v - out[h], axis=1) ** 2))
                    + 2.0 ** -18 * w @ norm(v, axis=1))
    return out, bound


def modest_pool(rng, S, Hkv):
    """(codes, scales) of k and of v whose rows differ little in size."""
    row = lambda: rng.standard_normal((S, Hkv, 64)) * np.exp(0.3 * rng.standard_normal((S, Hkv, 1)))  # noqa: E731
    return [*quantise(row()), *quantise(row())]


def unit_values(n, Hkv):
    """Value rows [n, Hkv, 64] in which each run of entries, as short as 64 Hkv runs
    allow, has one component to itself: with equal weights an output component is the
    run's entries counted, over n."""
    run = max(1, -(-n // (64 * Hkv)))
    slot = np.arange(n) // run
    v = np.zeros((n, Hkv, 64))
    v[np.arange(n), slot % Hkv, slot // Hkv] = 1
    return v


def flat_scores(seed, Hkv, n, size=256.0, q_pos=12345):
    """A query of large components and keys, at position 0, whose scores are all within
    1.5: (q [Hkv, 64] in bf16 values, q_pos, codes and scales of K [n, Hkv, 64])."""
    rng = np.random.default_rng(seed)
    q = size * rng.standard_normal((Hkv, 64))
    q = (q.astype(np.float32).view(np.uint32) & 0xffff0000).view(np.float32).astype(np.float64)
    qr = turn(q[None], [q_pos])[0]
    codes, scale = np.zeros((n, Hkv, 64), np.uint8), np.zeros((n, Hkv), np.uint8)
    for g in range(Hkv):
        have = 0
        while have < n:
            c, s = quantise(rng.standard_normal((40000, 64)))
            near = np.flatnonzero(np.abs(held(c, s) @ qr[g] / 8) < 1.5)[:n - have]
            codes[have:have + len(near), g], scale[have:have + len(near), g] = c[near], s[near]
            have += len(near)
    return q, q_pos, codes, scale
