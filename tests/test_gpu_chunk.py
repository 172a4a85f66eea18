"""A chunk of new tokens over the page-size-1 pool: row preparation, chunk
attention, attention mass and eviction by mass, against their definitions in
64 bits, and run one after the other as a serving step does.

Tolerances.  u = 2^-8 (bf16) or 2^-24 (fp32) is half a rounding step relative
to the value.  A score is a sum of 64 fp32 products: its error is at most
E = 2^-18 max_j sum_d |q_d k_jd| / 8 (64 additions of 2^-24 each, doubled for
tensor cores that truncate, doubled for the conversion to base 2), and a
weight's relative error is that of its score.
* out: |err| <= u |out| + (u + 2 E + 2^-18) A with A = sum_j p_j |v_j|: the
  stored rounding; bf16 also rounds each weight before the product with V
  (fp32: no such rounding, the term stays for simplicity: 2^-24); 2^-18 for
  the fp32 sums.
* lse: E + 2^-21 (1 + |lse|): the score's error, and the rounding of the
  maximum, of the sum (relative, so absolute in the logarithm) and of the
  result, a few 2^-24 each.
* mass: (2 E + 2^-18) times the mass: every term is positive.  A weight below
  2^-126 is no normal fp32 number and counts as 0: 2^-126 per term.
* prepared rows: u |y| + 2^-20 |row's largest pair|: angles are good to 4e-7
  and the norm and rotation to a few 2^-24.
"""
import numpy as np
import pytest

import kv_cache_drop_gb300 as akv
import oracle
import workloads

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _torch():
    import torch
    return torch


def _rand(rng, shape, dtype, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return workloads.bf16_bits(x) if dtype == "bf16" else x


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


# ---------------------------------------------------------------- the batch

class Batch:
    """Chunks of m_b rows over lists of n_b entries scattered in a pool;
    `lead` and `tail` rows of q that belong to no request."""

    def __init__(self, seed, m, n, Hq, Hkv, dtype, scale=1.0, spare=7, tail=0, S=None):
        rng = np.random.default_rng(seed)
        self.rng, self.m, self.n, self.Hq, self.Hkv, self.dtype = rng, m, n, Hq, Hkv, dtype
        self.B = len(m)
        self.q_ptr = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
        self.kv_ptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.S = S or int(self.kv_ptr[-1]) + spare
        self.rows = int(self.q_ptr[-1]) + tail
        self.idx = rng.permutation(self.S)[:int(self.kv_ptr[-1])].astype(np.int32)
        self.q = _rand(rng, (self.rows, Hq, 64), dtype, scale)
        self.k = _rand(rng, (self.S, Hkv, 64), dtype)
        self.v = _rand(rng, (self.S, Hkv, 64), dtype)
        self.shp = akv.shape(Hq, Hkv, 64, dtype)
        self.max_q, self.max_kv = max(m), max(n)

    def device(self):
        d = lambda x: akv.to_device(x, self.dtype)  # noqa: E731
        return dict(q=d(self.q), k=d(self.k), v=d(self.v), q_ptr=akv.i32_device(self.q_ptr),
                    kv_ptr=akv.i32_device(self.kv_ptr), idx=akv.i32_device(self.idx))

    def wide(self, x):
        return oracle.widen(x, self.dtype)

    def scores(self, b):
        """(scores [m, Hq, n] scaled, -inf where hidden; E [m, Hq])."""
        q = self.wide(self.q[self.q_ptr[b]:self.q_ptr[b + 1]])
        K = self.wide(self.k[self.idx[self.kv_ptr[b]:self.kv_ptr[b + 1]]])
        K = np.repeat(K, self.Hq // self.Hkv, axis=1)
        s = np.einsum("ihd,jhd->ihj", q, K) / 8
        size = np.einsum("ihd,jhd->ihj", np.abs(q), np.abs(K)) / 8
        seen = self.n[b] - self.m[b] + 1 + np.arange(self.m[b])
        hid = np.arange(self.n[b])[None, :] >= seen[:, None]
        s = np.where(hid[:, None, :], -np.inf, s)
        size = np.where(hid[:, None, :], 0, size)
        return s, 2.0 ** -18 * (size.max(-1) if self.n[b] else np.zeros(size.shape[:2]))

    def attend(self, b):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
        s, E = self.scores(b)
        V = np.repeat(self.wide(self.v[self.idx[self.kv_ptr[b]:self.kv_ptr[b + 1]]]),
                      self.Hq // self.Hkv, axis=1)
        empty = np.isneginf(s).all(-1)
        top = np.where(empty, 0, s.max(-1, initial=-np.inf))
        p = np.where(np.isneginf(s), 0, np.exp(s - top[..., None]))
        tot = np.where(empty, 1, p.sum(-1))
        p /= tot[..., None]
        out = np.einsum("ihj,jhd->ihd", p, V)
        A = np.einsum("ihj,jhd->ihd", p, np.abs(V))
        lse = np.where(empty, -np.inf, top + np.log(tot))
        u = U[self.dtype]
        tol = u * np.abs(out) + (u + 2 * E[..., None] + 2.0 ** -18) * A
        return out, lse, tol, E + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, lse)))

    def mass(self, b, lse, mass_in=None, decay=1.0):
        """(mass, tolerance) given fp32 lse rows of request b."""
        s, E = self.scores(b)
        l64 = lse.astype(np.float64)
        with np.errstate(invalid="ignore"):
            w = np.where(np.isneginf(s) | np.isneginf(l64)[..., None], 0, np.exp(s - l64[..., None]))
        got = w.sum((0, 1))
        tol = (2 * E.max(initial=0) + 2.0 ** -18) * got + 2.0 ** -126 * self.m[b] * self.Hq
        if mass_in is not None:
            old = decay * mass_in[:max(0, self.n[b] - self.m[b])].astype(np.float64)
            got[:len(old)] += old
            tol[:len(old)] += 2.0 ** -22 * np.abs(old)
        return got, tol


def run_chunk(bt, d, lse=True, fill=7.0, max_q=None, max_kv=None, stream=None):
    torch = _torch()
    max_q, max_kv = max_q or bt.max_q, bt.max_kv if max_kv is None else max_kv
    out = torch.full_like(d["q"], fill)
    l = torch.full((bt.rows, bt.Hq), fill, device="cuda") if lse else None
    ws = torch.empty(akv.akv_chunk_workspace(bt.shp, bt.B, bt.rows, max_q, max_kv),
                     dtype=torch.uint8, device="cuda")
    akv.akv_chunk_attention(bt.shp, bt.B, d["q_ptr"], d["q"], d["k"], d["v"], d["kv_ptr"],
                            d["idx"], max_q, max_kv, out, l, ws, stream=stream)
    return out, l


def check_chunk(bt, out, lse, fill=7.0):
    torch = _torch()
    torch.cuda.synchronize()
    o = _host(out)
    for b in range(bt.B):
        r = slice(bt.q_ptr[b], bt.q_ptr[b + 1])
        if not bt.m[b]:
            continue
        want, wl, tol, tl = bt.attend(b)
        err = np.abs(o[r] - want)
        assert np.all(err <= tol), (b, float((err / np.maximum(tol, 1e-30)).max()))
        if lse is not None:
            g = _host(lse)[r]
            none = np.isneginf(wl)
            assert np.array_equal(np.isneginf(g), none)
            err = np.abs(g[~none] - wl[~none])
            assert np.all(err <= tl[~none]), float((err / tl[~none]).max())
    assert np.all(o[bt.q_ptr[-1]:] == fill)  # rows of no request
    if lse is not None:
        assert np.all(_host(lse)[bt.q_ptr[-1]:] == fill)


def run_mass(bt, d, lse, mass_in, decay, out, max_q=None, max_kv=None):
    torch = _torch()
    max_q, max_kv = max_q or bt.max_q, bt.max_kv if max_kv is None else max_kv
    ws = torch.empty(akv.akv_attention_mass_workspace(bt.shp, bt.B, bt.rows, max_q, max_kv),
                     dtype=torch.uint8, device="cuda")
    akv.akv_attention_mass(bt.shp, bt.B, d["q_ptr"], d["q"], d["k"], d["kv_ptr"], d["idx"], max_q,
                           max_kv, lse, decay, mass_in, out, ws)


def check_mass(bt, lse, mass_in, decay, out, fill):
    torch = _torch()
    torch.cuda.synchronize()
    g, l, mi = _host(out), lse.cpu().numpy(), None if mass_in is None else mass_in.cpu().numpy()
    for b in range(bt.B):
        want, tol = bt.mass(b, l[bt.q_ptr[b]:bt.q_ptr[b + 1]], None if mi is None else mi[b], decay)
        err = np.abs(g[b, :bt.n[b]] - want)
        assert np.all(err <= tol), (b, float((err / np.maximum(tol, 1e-300)).max()))
        assert np.all(g[b, bt.n[b]:] == fill)  # behind the list: left as it was


# name: (chunk lengths, list lengths)
SHAPES = {
    "single tokens": ([1, 1, 1, 1], [1, 2, 129, 700]),
    "tile edges": ([15, 16, 17, 32, 33, 127, 128, 129], [15, 31, 300, 32, 64, 128, 129, 257]),
    "empty": ([0, 3, 0, 5, 1], [0, 3, 40, 2, 0]),          # rows that see nothing, empty chunks
    "one long": ([2], [9000]),
    "uneven": ([1, 200, 3, 64], [5000, 200, 1000, 65]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 4), (24, 3), (2, 2), (32, 16), (20, 1)])
@pytest.mark.parametrize("name", list(SHAPES))
def test_chunk_attention_and_mass(name, Hq, Hkv, dtype):
    torch = _torch()
    m, n = SHAPES[name]
    bt = Batch(100 + len(name) + Hq, m, n, Hq, Hkv, dtype, tail=3)
    d = bt.device()
    out, lse = run_chunk(bt, d)
    check_chunk(bt, out, lse)
    rng = np.random.default_rng(5)
    mass_in = torch.from_numpy(rng.random((bt.B, bt.max_kv)).astype(np.float32)).cuda()
    for mi, decay in ((None, 1.0), (mass_in, 0.5)):
        got = torch.full((bt.B, bt.max_kv), -3.0, device="cuda")
        run_mass(bt, d, lse, mi, decay, got)
        check_mass(bt, lse, mi, decay, got, -3.0)


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (100, 2), (12, 4), (9, 3)])
def test_chunk_other_groups(Hq, Hkv):
    """Groups that fill a row tile, that do not divide one, and odd ones."""
    torch = _torch()
    bt = Batch(7, [1, 40, 9], [300, 700, 9], Hq, Hkv, "bf16")
    d = bt.device()
    out, lse = run_chunk(bt, d)
    check_chunk(bt, out, lse)
    got = torch.zeros(bt.B, bt.max_kv, device="cuda")
    run_mass(bt, d, lse, None, 1.0, got)
    check_mass(bt, lse, None, 1.0, got, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [([1, 1], [20000, 700]), ([6], [9000]), ([10, 3], [6000, 5999]),
                                 ([40, 30], [9001, 130]), ([300, 2], [9000, 8000])])
def test_chunk_long_lists(m, n, dtype):
    """Few rows over long lists: the lists are cut into splits (for 16 query
    heads over 4 KV heads, every form of the kernels), some rows' entries
    within one split and some over several, and the mass of an entry shared
    by several CTAs."""
    torch = _torch()
    bt = Batch(13, m, n, 16, 4, dtype)
    d = bt.device()
    out, lse = run_chunk(bt, d)
    check_chunk(bt, out, lse)
    again, lse2 = run_chunk(bt, d)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # no order of atomics in it
    got, got2 = (torch.zeros(bt.B, bt.max_kv, device="cuda") for _ in range(2))
    run_mass(bt, d, lse, None, 1.0, got)
    check_mass(bt, lse, None, 1.0, got, 0.0)
    run_mass(bt, d, lse, None, 1.0, got2)
    assert torch.equal(got, got2)


def test_chunk_many_requests():
    """300 requests of a few rows each, every seventh without any."""
    rng = np.random.default_rng(14)
    m = [0 if b % 7 == 3 else int(rng.integers(1, 4)) for b in range(300)]
    n = [int(rng.integers(0, 60)) for _ in range(300)]
    torch = _torch()
    for shift in (0, 30):  # 30: chunks long enough for the other kernels
        bt = Batch(15, [x + shift if x else 0 for x in m], [x + shift for x in n], 8, 2, "bf16")
        d = bt.device()
        out, lse = run_chunk(bt, d)
        check_chunk(bt, out, lse)
        got = torch.zeros(bt.B, bt.max_kv, device="cuda")
        run_mass(bt, d, lse, None, 1.0, got)
        check_mass(bt, lse, None, 1.0, got, 0.0)


@pytest.mark.parametrize("m,dtype", [(1, "bf16"), (10, "bf16"), (40, "bf16"), (150, "bf16"), (40, "f32")])
def test_no_wait_gave_up(m, dtype):
    """The status word that the tensor-core kernels' bounded waits would set
    reads 0 after a call, whatever the workspace held before."""
    torch = _torch()
    bt = Batch(16, [m, m], [700, 300], 16, 4, dtype)
    d = bt.device()
    out, lse = torch.empty_like(d["q"]), torch.empty(bt.rows, 16, device="cuda")
    ws = torch.full((akv.akv_chunk_workspace(bt.shp, 2, bt.rows, m, 700),), 255, dtype=torch.uint8,
                    device="cuda")
    akv.akv_chunk_attention(bt.shp, 2, d["q_ptr"], d["q"], d["k"], d["v"], d["kv_ptr"], d["idx"], m,
                            700, out, lse, ws)
    assert akv.akv_workspace_status(ws) == 0
    check_chunk(bt, out, lse)
    ws = torch.full((akv.akv_attention_mass_workspace(bt.shp, 2, bt.rows, m, 700),), 255,
                    dtype=torch.uint8, device="cuda")
    got = torch.zeros(2, 700, device="cuda")
    akv.akv_attention_mass(bt.shp, 2, d["q_ptr"], d["q"], d["k"], d["kv_ptr"], d["idx"], m, 700, lse,
                           1.0, None, got, ws)
    assert akv.akv_workspace_status(ws) == 0
    check_mass(bt, lse, None, 1.0, got, 0.0)


def test_no_lists_at_all():
    """max_kv = 0 with no pool: rows get zeros and -inf."""
    torch = _torch()
    for dtype in ("bf16", "f32"):
        for m in (1, 40, 300):
            shp = akv.shape(16, 4, 64, dtype)
            q = akv.to_device(_rand(np.random.default_rng(1), (m, 16, 64), dtype), dtype)
            pool = q.new_zeros(0, 4, 64)
            out, lse = torch.full_like(q, 7.0), torch.zeros(m, 16, device="cuda")
            ws = torch.empty(akv.akv_chunk_workspace(shp, 1, m, m, 0), dtype=torch.uint8, device="cuda")
            akv.akv_chunk_attention(shp, 1, akv.i32_device([0, m]), q, pool, pool, akv.i32_device([0, 0]),
                                    akv.i32_device([]), m, 0, out, lse, ws)
            torch.cuda.synchronize()
            assert not out.any() and bool(torch.isneginf(lse).all())


def test_mass_of_a_long_chunk():
    """Each entry's mass is the sum of 16,000 weights (1,000 rows of 16 heads
    over 1,100 entries): the additions' roundings do not add up."""
    torch = _torch()
    bt = Batch(17, [1000], [1100], 16, 4, "bf16")
    d = bt.device()
    _, lse = run_chunk(bt, d)
    got = torch.zeros(1, 1100, device="cuda")
    run_mass(bt, d, lse, None, 1.0, got)
    check_mass(bt, lse, None, 1.0, got, 0.0)
    want, _ = bt.mass(0, lse.cpu().numpy())
    g = _host(got)[0]
    # in one fp32 chain 16,000 additions would be off by about sqrt(16000)
    # 2^-25 = 4e-6; a score's own error is a few 2^-24 of its size, 1e-6 of a
    # weight here
    assert np.linalg.norm(g - want) / np.linalg.norm(want) < 2e-6
    assert abs(g.sum() / (1000 * 16) - 1) < 2e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 4, 300])
def test_chunk_peaky_scores(m, dtype):
    """Scores of standard deviation 16: sharp rows, running maxima that rise."""
    bt = Batch(8, [m, m], [1500, 333], 16, 4, dtype, scale=16)
    d = bt.device()
    out, lse = run_chunk(bt, d)
    check_chunk(bt, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 10, 40, 300])
def test_chunk_scores_that_jump(m, dtype):
    """Scores that rise by 60 to 190 within one window after hundreds of low
    ones, rise in steps, or fall from the first entry on: weights relative to
    anything but the running maximum would overflow or vanish."""
    n = 1500
    for case in ("one peak", "late peak", "steps", "sink", "two levels"):
        bt = Batch(18, [m], [n], 16, 4, dtype)
        level = np.zeros(n)
        if case == "one peak":
            level[:] = -3
            level[700] = 3
        elif case == "late peak":
            level[:] = -3
            level[n - m] = 3          # every row sees it
            level[1100:1110] = 1
        elif case == "steps":
            level = -3 + np.floor(np.arange(n) / 100) * 0.4
        elif case == "sink":
            level[0] = 3
        else:
            level[:400], level[400:] = -2, 2
        rng = np.random.default_rng(19)
        k = (level[:, None, None] + 0.05 * rng.standard_normal((n, 4, 64))).astype(np.float32)
        q = (4 + 0.05 * rng.standard_normal((m, 16, 64))).astype(np.float32)  # scores 32 x level
        pool = np.zeros((bt.S, 4, 64), np.float32)
        pool[bt.idx] = k
        bt.q, bt.k = (workloads.bf16_bits(x) if dtype == "bf16" else x for x in (q, pool))
        d = bt.device()
        out, lse = run_chunk(bt, d)
        check_chunk(bt, out, lse)
        got = _torch().zeros(1, n, device="cuda")
        run_mass(bt, d, lse, None, 1.0, got)
        check_mass(bt, lse, None, 1.0, got, 0.0)


@pytest.mark.parametrize("B,m,n", [(80, 30, 1500), (44, 40, 1500)])
def test_chunk_scores_that_jump_late(B, m, n):
    """A jump after a thousand entries of an unsplit list: the pass with exact
    maxima starts over and walks the whole list again, every ring of copies
    several times round."""
    bt = Batch(20, [m] * B, [n] * B, 16, 4, "bf16")
    rng = np.random.default_rng(21)
    pool = np.zeros((bt.S, 4, 64), np.float32)
    for b in range(B):
        level = np.full(n, -3.0)
        level[1200 + b % 97] = 2 + (b % 3) / 2
        if b % 4 == 1:
            level[: 200 + b] = -1.5
        pool[bt.idx[bt.kv_ptr[b]:bt.kv_ptr[b + 1]]] = level[:, None, None] + 0.05 * rng.standard_normal((n, 4, 64))
    q = (4 + 0.05 * rng.standard_normal((m * B, 16, 64))).astype(np.float32)
    bt.q, bt.k = workloads.bf16_bits(q), workloads.bf16_bits(pool)
    d = bt.device()
    out, lse = run_chunk(bt, d)
    check_chunk(bt, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [500, 4000])
@pytest.mark.parametrize("m", [2, 10, 40, 300])
def test_hidden_entries_do_not_reach_a_row(m, more, dtype):
    """NaN and infinities in the value and key of a chunk's later tokens, and
    in pool rows that no list names (row 0 among them): earlier rows keep
    their values, and rows that see such an entry show it."""
    torch = _torch()
    n = m + more
    bt = Batch(9, [m, m], [n, m], 16, 4, dtype, spare=50)
    clean = Batch(9, [m, m], [n, m], 16, 4, dtype, spare=50)
    d = bt.device()
    listed = np.zeros(bt.S, bool)
    listed[bt.idx] = True
    bad_rows = torch.from_numpy(np.flatnonzero(~listed)).cuda()
    d["k"][bad_rows] = float("nan")
    d["v"][bad_rows] = float("nan")
    cut = m // 2
    # request 0: V of token `cut` has a NaN and an infinity; request 1: K of
    # token `cut` is NaN
    at0, at1 = int(bt.idx[n - m + cut]), int(bt.idx[bt.kv_ptr[1] + cut])
    d["v"][at0, 0, 3] = float("nan")
    d["v"][at0, 1, 5] = float("inf")
    d["v"][at0, 2, 7] = -float("inf")
    d["k"][at1, 0] = float("nan")
    out, lse = run_chunk(bt, d)
    torch.cuda.synchronize()
    o = _host(out)
    want, _, tol, _ = clean.attend(0)
    w1, _, t1, _ = clean.attend(1)
    G = 4
    assert np.all(np.abs(o[:cut] - want[:cut]) <= tol[:cut])
    late = o[cut:m]
    assert np.all(np.isnan(late[:, :G, 3])) and np.all(late[:, G:2 * G, 5] == np.inf)
    assert np.all(late[:, 2 * G:3 * G, 7] == -np.inf)
    rest = np.ones((m - cut, 16, 64), bool)
    rest[:, :G, 3] = rest[:, G:2 * G, 5] = rest[:, 2 * G:3 * G, 7] = False
    assert np.all((np.abs(late - want[cut:]) <= tol[cut:])[rest])
    o1 = o[m:]
    assert np.all(np.abs(o1[:cut] - w1[:cut]) <= t1[:cut])
    assert np.all(np.isnan(o1[cut:, :G]))
    assert np.all((np.abs(o1[cut:, G:] - w1[cut:, G:]) <= t1[cut:, G:]))
    assert np.all(np.isnan(_host(lse)[m + cut:, :G]))


def test_chunk_bounds_hold():
    """Pool indices outside [0, S) read row 0; chunks and lists longer than
    the given bounds, and row pointers past q, are cut: nothing outside the
    buffers is touched, and other requests keep their results."""
    torch = _torch()
    for dtype in ("f32", "bf16"):
        for m in (2, 40):
            bt = Batch(10, [m, m], [600, 300], 16, 4, dtype, tail=2)
            bt.idx[5], bt.idx[17], bt.idx[599] = -1, bt.S, 2**31 - 1
            d = bt.device()
            bt.idx[5] = bt.idx[17] = bt.idx[599] = 0
            out, lse = run_chunk(bt, d)
            check_chunk(bt, out, lse)
            got = torch.full((2, 600), -3.0, device="cuda")
            run_mass(bt, d, lse, None, 1.0, got)
            check_mass(bt, lse, None, 1.0, got, -3.0)
            # the last pointer runs past the rows: request 1's chunk is cut to them
            d["q_ptr"] = akv.i32_device([0, m, 10**6])
            out, lse = run_chunk(bt, d, max_q=m)
            torch.cuda.synchronize()
            want, _, tol, _ = bt.attend(0)
            assert np.all(np.abs(_host(out)[:m] - want) <= tol)


def test_chunk_equals_decode_and_prefill():
    """A chunk of one row is a decode step, and chunks of an empty cache are
    the rows of a restoration: the three paths of the library agree."""
    torch = _torch()
    r = workloads.random_request(3, n_msgs=1, max_len=200, Hq=16, Hkv=4, dtype="bf16",
                                 p_drop=0, p_repos=0, min_len=200)
    T, shp = r.T, akv.shape(16, 4, 64, "bf16")
    q, k, v = (akv.to_device(x, "bf16") for x in (r.q, r.k, r.v))
    slot = akv.i32_device(np.random.default_rng(1).permutation(T))
    pos = akv.i32_device(np.arange(T))
    kp, vp, qr = torch.zeros_like(k), torch.zeros_like(v), torch.empty_like(q)
    akv.akv_qk_norm_append(shp, T, q, k, v, pos, slot, kp, vp, qr,
                           flags=akv.AKV_ROPE_Q | akv.AKV_ROPE_K)
    kp2, vp2 = torch.zeros_like(k), torch.zeros_like(v)
    akv.akv_append_kv(shp, T, k, v, pos, slot, kp2, vp2)
    torch.cuda.synchronize()
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2)  # the same rotation
    ref, _ = oracle.replay_attention(*r.ops(), r.q, r.k, r.v, "bf16", r.rope_base)
    got = torch.empty_like(q)
    for a, b in ((0, 150), (150, 199), (199, 200)):  # three chunks
        m = b - a
        args = (shp, 1, akv.i32_device([0, m]), qr[a:b].contiguous(), kp, vp,
                akv.i32_device([0, b]), slot[:b].contiguous(), m, b)
        ws = torch.empty(akv.akv_chunk_workspace(shp, 1, m, m, b), dtype=torch.uint8, device="cuda")
        o = torch.empty(m, 16, 64, dtype=torch.bfloat16, device="cuda")
        akv.akv_chunk_attention(*args, o, None, ws)
        got[a:b] = o
    dec = torch.empty(1, 16, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(akv.akv_decode_workspace(shp, 1, T), dtype=torch.uint8, device="cuda")
    akv.akv_decode_attention(shp, 1, q[T - 1:].contiguous(), akv.i32_device([T - 1]), kp, vp,
                             akv.i32_device([0, T]), slot, T, dec, ws)
    torch.cuda.synchronize()
    from _util import assert_close
    assert_close(_host(got), ref, "bf16")
    assert_close(_host(dec), _host(got[T - 1:]), "bf16")


def test_chunk_long_pool_offsets():
    """Slots whose byte and element offsets pass 32 bits (a pool of 4.3
    million tokens, 8 KV heads)."""
    torch = _torch()
    S, Hq, Hkv = 4_300_000, 64, 8
    rng = np.random.default_rng(11)
    for m in (1, 40):
        n = 600
        bt = Batch(12, [m], [n], Hq, Hkv, "bf16")
        d = bt.device()
        k = torch.zeros(S, Hkv, 64, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros(S, Hkv, 64, dtype=torch.bfloat16, device="cuda")
        far = np.sort(rng.choice(np.arange(S - 5000, S), size=n, replace=False)).astype(np.int32)
        ft = torch.from_numpy(far.astype(np.int64)).cuda()
        old = torch.from_numpy(bt.idx.astype(np.int64)).cuda()
        k[ft], v[ft] = d["k"][old], d["v"][old]
        d["k"], d["v"], d["idx"] = k, v, akv.i32_device(far)
        out, lse = run_chunk(bt, d)
        check_chunk(bt, out, lse)
        got = torch.zeros(1, n, device="cuda")
        run_mass(bt, d, lse, None, 1.0, got)
        check_mass(bt, lse, None, 1.0, got, 0.0)
        # the append reaches them too
        qo = torch.empty(n, Hq, 64, dtype=torch.bfloat16, device="cuda")
        kn, vn = d["k"][ft].clone(), torch.randn(n, Hkv, 64, device="cuda").bfloat16()
        akv.akv_qk_norm_append(bt.shp, n, qo.zero_(), kn, vn, None, d["idx"], k, v, qo, flags=0)
        assert torch.equal(v[ft], vn) and torch.equal(k[ft], kn)
        del k, v, d


# ------------------------------------------------------------ preparation

def _prepared(x, w, pos, norm, rope, eps, dtype):
    y = oracle.widen(x, dtype)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (1 if w is None else w.astype(np.float64))
    return oracle.rope(y, pos[:, None], 10000.0) if rope else y


def _close_rows(got, want, dtype):
    h = want.shape[-1] // 2
    pair = np.sqrt(want[..., :h] ** 2 + want[..., h:] ** 2).max(-1, keepdims=True)
    err, tol = np.abs(got - want), U[dtype] * np.abs(want) + 2.0 ** -20 * pair
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 4), (24, 3), (2, 2), (5, 5), (20, 1)])
@pytest.mark.parametrize("n", [1, 14, 333])
def test_qk_norm_append(n, Hq, Hkv, dtype):
    torch = _torch()
    rng = np.random.default_rng(n + Hq)
    shp = akv.shape(Hq, Hkv, 64, dtype)
    x = _rand(rng, (n, Hq + 2 * Hkv, 64), dtype, 3.0)
    if n > 5:
        x[3] = 0  # rows of zeros: the norm's eps
    S = n + 20
    slot = rng.permutation(S)[:n].astype(np.int32)
    pad = np.zeros(n, bool)
    if n > 1:
        pad[n // 2::5] = True
        slot[pad] = np.where(np.arange(pad.sum()) % 2, -1, S + 7)
    pos = rng.integers(-5, 300_000, size=n).astype(np.int32)  # past 2^18, and below zero
    qw, kw = (1 + 0.3 * rng.standard_normal(64)).astype(np.float32), None
    kp0, vp0 = _rand(rng, (S, Hkv, 64), dtype), _rand(rng, (S, Hkv, 64), dtype)
    fused = akv.to_device(x, dtype)
    blocks = [fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]]
    xs = [x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]]
    for flags in (15, 0, akv.AKV_NORM_Q | akv.AKV_ROPE_K, akv.AKV_NORM_K | akv.AKV_ROPE_Q,
                  akv.AKV_NORM_Q | akv.AKV_NORM_K):
        for strided in (True, False):
            q, k, v = blocks if strided else [t.contiguous() for t in blocks]
            kp, vp = akv.to_device(kp0, dtype), akv.to_device(vp0, dtype)
            qo = torch.full((n, Hq, 64), 7.0, dtype=kp.dtype, device="cuda")
            akv.akv_qk_norm_append(shp, n, q, k, v, akv.i32_device(pos), akv.i32_device(slot), kp, vp,
                                   qo, q_weight=torch.from_numpy(qw).cuda(), k_weight=kw, eps=1e-5,
                                   flags=flags)
            torch.cuda.synchronize()
            ok = ~pad
            wq = _prepared(xs[0], qw, pos, flags & 1, flags & 4, 1e-5, dtype)
            wk = _prepared(xs[1], kw, pos, flags & 2, flags & 8, 1e-5, dtype)
            _close_rows(_host(qo)[ok], wq[ok], dtype)
            assert np.all(_host(qo)[pad] == 7.0)  # padding rows: left as they were
            gk, gv = _host(kp), _host(vp)
            _close_rows(gk[slot[ok]], wk[ok], dtype)
            assert np.array_equal(gv[slot[ok]], oracle.widen(xs[2], dtype)[ok])
            other = np.ones(S, bool)
            other[slot[ok]] = False
            assert np.array_equal(gk[other], oracle.widen(kp0, dtype)[other])
            assert np.array_equal(gv[other], oracle.widen(vp0, dtype)[other])
    # in place
    q = blocks[0].contiguous()
    akv.akv_qk_norm_append(shp, n, q, blocks[1], blocks[2], akv.i32_device(pos),
                           akv.i32_device(slot), kp, vp, q, eps=1e-5)
    torch.cuda.synchronize()
    _close_rows(_host(q)[ok], _prepared(xs[0], None, pos, 1, 1, 1e-5, dtype)[ok], dtype)
    assert np.array_equal(_host(q)[pad], oracle.widen(xs[0], dtype)[pad])


def test_qk_norm_append_many_rows():
    """More than 2^31 elements of q (540,000 tokens of 64 heads): the last
    tokens' rows are right."""
    torch = _torch()
    n, Hq, Hkv = 540_000, 64, 1
    shp = akv.shape(Hq, Hkv, 64, "bf16")
    q = torch.zeros(n, Hq, 64, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(2)
    tail = _rand(rng, (5, Hq, 64), "bf16")
    q[-5:] = akv.to_device(tail, "bf16")
    k = torch.zeros(n, Hkv, 64, dtype=torch.bfloat16, device="cuda")
    kp, vp = torch.empty_like(k), torch.empty_like(k)
    slot = torch.arange(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    akv.akv_qk_norm_append(shp, n, q, k, k, pos, slot, kp, vp, q)
    torch.cuda.synchronize()
    want = _prepared(tail, None, np.arange(n - 5, n), True, True, 1e-6, "bf16")
    _close_rows(_host(q[-5:]), want, "bf16")


# --------------------------------------------------------------- eviction

def _evict_ref(mass, n, keep, n_first, n_recent):
    """Kept list positions of one request, ascending."""
    key = np.where(np.isnan(mass[:n]), -np.inf, mass[:n].astype(np.float64))
    key[:n_first] = np.inf
    key[max(0, n - n_recent):] = np.inf
    order = np.lexsort((np.arange(n), -key))
    return np.sort(order[:min(max(keep, 0), n)])


def _run_evict(lens, mass, keep, n_first, n_recent, with_pos=True, max_kv=None, caps=None, seed=0):
    torch = _torch()
    rng = np.random.default_rng(seed)
    B, ptr = len(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    nnz = int(ptr[-1])
    idx = rng.permutation(nnz + 5)[:nnz].astype(np.int32)
    pos = rng.integers(0, 1 << 20, size=nnz).astype(np.int32)
    max_kv = max(lens) if max_kv is None else max_kv
    full = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    cap, dcap, stride = caps or (nnz + 3, nnz + 3, mass.shape[1])
    o = dict(ptr=full(B + 1), idx=full(cap), pos=full(cap) if with_pos else None,
             mass=torch.full((B, stride), -9.0, device="cuda"), dptr=full(B + 1), drop=full(dcap))
    akv.akv_evict_by_mass(B, akv.i32_device(ptr), akv.i32_device(idx),
                          akv.i32_device(pos) if with_pos else None, max_kv,
                          torch.from_numpy(mass).cuda(), akv.i32_device(keep), n_first, n_recent,
                          o["ptr"], o["idx"], o["pos"], o["mass"], o["dptr"], o["drop"])
    torch.cuda.synchronize()
    o = {k: None if t is None else t.cpu().numpy() for k, t in o.items()}
    kp, dp = 0, 0
    for b, n in enumerate(lens):
        kept = _evict_ref(mass[b], n, keep[b], n_first, n_recent)
        drop = np.setdiff1d(np.arange(n), kept)
        assert o["ptr"][b] == kp and o["dptr"][b] == dp
        put = lambda dst, at, x: np.testing.assert_array_equal(  # noqa: E731
            dst[at:at + len(x)], x[:max(0, len(dst) - at)])
        put(o["idx"], kp, idx[ptr[b] + kept])
        if with_pos:
            put(o["pos"], kp, pos[ptr[b] + kept])
        put(o["drop"], dp, idx[ptr[b] + drop])
        np.testing.assert_array_equal(o["mass"][b, :len(kept)], mass[b, kept][:stride])
        assert np.all(o["mass"][b, len(kept):] == -9)
        kp, dp = kp + len(kept), dp + len(drop)
    assert o["ptr"][-1] == kp and o["dptr"][-1] == dp
    assert np.all(o["idx"][kp:] == -9) and np.all(o["drop"][dp:] == -9)


@pytest.mark.parametrize("lens", [[1], [0, 0], [1, 2, 3, 0, 31, 32, 33], [127, 128, 129, 4095],
                                  [16384, 16383], [16385, 1], [20000, 5, 70001], [131_072, 131_071],
                                  [131_073], [300_000], [140_000] + [7] * 9, [3] * 200])
def test_evict_sizes(lens):
    rng = np.random.default_rng(sum(lens))
    mass = np.exp(2 * rng.standard_normal((len(lens), max(max(lens), 1)))).astype(np.float32)
    for frac in (0.0, 0.3, 0.999, 1.5):
        keep = [int(frac * n) for n in lens]
        _run_evict(lens, mass, keep, 0, 0)
        _run_evict(lens, mass, keep, 4, 16, with_pos=False)


def test_evict_ties_and_special_masses():
    """Equal masses go by list position; zeros of both signs tie; infinities,
    negative values, subnormals and NaN have their place; more protected
    entries than the budget; budgets below zero."""
    rng = np.random.default_rng(3)
    n = 5000
    flat = np.full((1, n), 0.25, np.float32)
    few = rng.integers(0, 3, size=(1, n)).astype(np.float32)
    odd = rng.choice(np.array([0.0, -0.0, np.inf, -np.inf, np.nan, -np.nan, 1e-42, -1e-42, 1.0, -1.0,
                               3.4e38, -3.4e38], np.float32), size=(1, n))
    for mass in (flat, few, odd):
        for keep in (1, 17, 1234, 4999, 5000, 9999, 0, -3):
            _run_evict([n], mass, [keep], 0, 0)
            _run_evict([n], mass, [keep], 40, 100)
    _run_evict([n], few, [50], 2**31 - 1, 2**31 - 1)  # all protected
    _run_evict([n, n], np.concatenate([few, odd]), [100, 200], 150, 150)


def test_evict_bounds_hold():
    """Outputs shorter than the result are filled to their end and no
    further; a list longer than max_kv is cut to it."""
    rng = np.random.default_rng(4)
    lens = [1000, 700]
    mass = rng.random((2, 1000)).astype(np.float32)
    _run_evict(lens, mass, [400, 300], 1, 1, caps=(500, 600, 350))
    torch = _torch()
    out = torch.full((2000,), -9, dtype=torch.int32, device="cuda")
    p, dp = (torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(2))
    om = torch.empty(1, 100, device="cuda")
    akv.akv_evict_by_mass(1, akv.i32_device([0, 1000]), akv.i32_device(np.arange(1000)), None, 100,
                          torch.from_numpy(mass[:1, :100].copy()).cuda(), akv.i32_device([60]), 0, 0,
                          p, out, None, om, dp, out[1000:])
    torch.cuda.synchronize()
    assert p.tolist() == [0, 60] and dp.tolist() == [0, 40]
    np.testing.assert_array_equal(out[:60].cpu().numpy(), _evict_ref(mass[0], 100, 60, 0, 0))


# ------------------------------------------------------------- as one run

def _step(bt, t, flags=15):
    """prepare + append -> attention -> mass -> eviction, on the current stream."""
    akv.akv_qk_norm_append(bt.shp, bt.rows, t["x"][:, :bt.Hq], t["x"][:, bt.Hq:bt.Hq + bt.Hkv],
                           t["x"][:, bt.Hq + bt.Hkv:], t["pos"], t["slot"], t["k"], t["v"], t["q"],
                           q_weight=t["qw"], k_weight=t["kw"], flags=flags)
    akv.akv_chunk_attention(bt.shp, bt.B, t["q_ptr"], t["q"], t["k"], t["v"], t["kv_ptr"], t["idx"],
                            bt.max_q, bt.max_kv, t["out"], t["lse"], t["ws"])
    akv.akv_attention_mass(bt.shp, bt.B, t["q_ptr"], t["q"], t["k"], t["kv_ptr"], t["idx"], bt.max_q,
                           bt.max_kv, t["lse"], 0.5, t["mass"], t["mass"], t["ws2"])
    akv.akv_evict_by_mass(bt.B, t["kv_ptr"], t["idx"], t["kv_pos"], bt.max_kv, t["mass"], t["keep"],
                          2, 4, t["o_ptr"], t["o_idx"], t["o_pos"], t["o_mass"], t["d_ptr"],
                          t["drop"])


def _step_tensors(bt, seed):
    torch = _torch()
    rng = np.random.default_rng(seed)
    d = bt.device()
    nnz = int(bt.kv_ptr[-1])
    x = _rand(rng, (bt.rows, bt.Hq + 2 * bt.Hkv, 64), bt.dtype, 2.0)
    slot, pos, kv_pos = np.full(bt.rows, -1, np.int32), np.zeros(bt.rows, np.int32), np.zeros(nnz, np.int32)
    for b in range(bt.B):
        own = slice(bt.kv_ptr[b + 1] - bt.m[b], bt.kv_ptr[b + 1])
        r = slice(bt.q_ptr[b], bt.q_ptr[b + 1])
        kv_pos[bt.kv_ptr[b]:bt.kv_ptr[b + 1]] = np.sort(rng.choice(4 * bt.n[b] + 1, bt.n[b], False))
        slot[r], pos[r] = bt.idx[own], kv_pos[own]
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    size = akv.akv_chunk_workspace, akv.akv_attention_mass_workspace
    ws = [torch.empty(s(bt.shp, bt.B, bt.rows, bt.max_q, bt.max_kv), dtype=torch.uint8,
                      device="cuda") for s in size]
    d.update(x=akv.to_device(x, bt.dtype), pos=akv.i32_device(pos), slot=akv.i32_device(slot),
             kv_pos=akv.i32_device(kv_pos), qw=f(1 + 0.2 * rng.standard_normal(64)),
             kw=f(1 + 0.2 * rng.standard_normal(64)), out=torch.zeros_like(d["q"]),
             lse=torch.zeros(bt.rows, bt.Hq, device="cuda"), ws=ws[0], ws2=ws[1],
             mass=f(rng.random((bt.B, bt.max_kv))),
             keep=akv.i32_device([max(1, n // 2) for n in bt.n]), o_ptr=z(bt.B + 1), o_idx=z(nnz),
             o_pos=z(nnz), o_mass=torch.zeros(bt.B, bt.max_kv, device="cuda"), d_ptr=z(bt.B + 1),
             drop=z(nnz))
    d["x_host"], d["pos_host"], d["kv_pos_host"] = x, pos, kv_pos
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [[1, 1, 1], [3, 150, 1]])
def test_serving_run(m, dtype):
    """The four calls one after the other, each checked against 64 bits on
    what the call before it left; then a decode over the kept lists, and a
    repos of one of them."""
    torch = _torch()
    bt = Batch(21, m, [400, 900, 33], 16, 4, dtype)
    t = _step_tensors(bt, 22)
    mass0 = t["mass"].clone()
    _step(bt, t)
    torch.cuda.synchronize()
    # what the preparation left
    qw, kw = t["qw"].cpu().numpy(), t["kw"].cpu().numpy()
    x = t["x_host"]
    _close_rows(_host(t["q"]), _prepared(x[:, :16], qw, t["pos_host"], 1, 1, 1e-6, dtype), dtype)
    own = np.concatenate([np.arange(bt.kv_ptr[b + 1] - bt.m[b], bt.kv_ptr[b + 1]) for b in range(3)])
    _close_rows(_host(t["k"])[bt.idx[own]], _prepared(x[:, 16:20], kw, t["pos_host"], 1, 1, 1e-6, dtype),
                dtype)
    raw = lambda a: (a.view(torch.int16).cpu().numpy().view(np.uint16) if dtype == "bf16"  # noqa: E731
                     else a.cpu().numpy())
    bt.q, bt.k, bt.v = raw(t["q"]), raw(t["k"]), raw(t["v"])
    check_chunk(bt, t["out"], t["lse"])
    l, g = t["lse"].cpu().numpy(), t["mass"].cpu().numpy()
    for b in range(3):
        want, tol = bt.mass(b, l[bt.q_ptr[b]:bt.q_ptr[b + 1]], mass0[b].cpu().numpy(), 0.5)
        assert np.all(np.abs(g[b, :bt.n[b]] - want) <= tol)
    o_ptr = t["o_ptr"].cpu().numpy()
    for b in range(3):
        kept = _evict_ref(g[b], bt.n[b], max(1, bt.n[b] // 2), 2, 4)
        sl = slice(o_ptr[b], o_ptr[b + 1])
        np.testing.assert_array_equal(t["o_idx"].cpu().numpy()[sl], bt.idx[bt.kv_ptr[b] + kept])
        np.testing.assert_array_equal(t["o_pos"].cpu().numpy()[sl], t["kv_pos_host"][bt.kv_ptr[b] + kept])
    # the next decode reads the kept lists as they are
    q = akv.to_device(_rand(bt.rng, (3, 16, 64), dtype), dtype)
    qpos = akv.i32_device([int(t["kv_pos_host"].max()) + 1] * 3)
    dec = torch.empty_like(q)
    wsd = torch.empty(akv.akv_decode_workspace(bt.shp, 3, bt.max_kv), dtype=torch.uint8, device="cuda")
    akv.akv_decode_attention(bt.shp, 3, q, qpos, t["k"], t["v"], t["o_ptr"], t["o_idx"], bt.max_kv, dec,
                             wsd)
    torch.cuda.synchronize()
    ref = oracle.decode_attention(raw(q), qpos.cpu().numpy(), bt.k, bt.v, o_ptr,
                                  t["o_idx"].cpu().numpy()[:o_ptr[-1]], dtype, 10000.0)
    from _util import assert_close
    assert_close(_host(dec), ref, dtype)
    # and a repos renumbers request 1's kept entries 0 .. r-1
    r = int(o_ptr[2] - o_ptr[1])
    src, pf = t["o_idx"][o_ptr[1]:o_ptr[2]].contiguous(), t["o_pos"][o_ptr[1]:o_ptr[2]].contiguous()
    ko = torch.empty(r, 4, 64, dtype=t["k"].dtype, device="cuda")
    vo = torch.empty_like(ko)
    akv.akv_repos_rotate(bt.shp, r, src, pf, None, t["k"], t["v"], ko, vo)
    torch.cuda.synchronize()
    want = oracle.rope(bt.wide(bt.k)[src.cpu().numpy()], (np.arange(r) - pf.cpu().numpy())[:, None], 10000.0)
    _close_rows(_host(ko), want, dtype)


@pytest.mark.parametrize("m", [[1, 1, 1], [3, 150, 1]])
def test_serving_run_captured(m):
    """The four calls captured once and replayed for another batch of other
    lengths within the bounds: the same as calling them eagerly, bit for bit.
    The eager calls of the second batch run on another stream."""
    torch = _torch()
    a = Batch(31, m, [400, 900, 33], 16, 4, "bf16")
    b = Batch(32, [1, 1, 1] if max(m) == 1 else [100, 20, 34], [900, 200, 233], 16, 4, "bf16", S=a.S)
    b.max_q, b.max_kv = a.max_q, a.max_kv
    ta, tb = _step_tensors(a, 33), _step_tensors(b, 34)
    mass_a, mass_b = ta["mass"].clone(), tb["mass"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(a, ta)  # warm-up of the modules, and batch a's eager results
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = {k: ta[k].clone() for k in ("q", "out", "lse", "mass", "o_ptr", "o_idx", "o_pos", "o_mass")}
    with torch.cuda.stream(side):
        _step(b, tb)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    ta["mass"].copy_(mass_a)
    with torch.cuda.graph(g):
        _step(a, ta)
    g.replay()
    torch.cuda.synchronize()
    for k, want in first.items():
        assert torch.equal(ta[k], want), k
    # batch b in the captured buffers
    rows, nnz = b.rows, int(b.kv_ptr[-1])
    ta["mass"].copy_(mass_b)
    ta["x"][:rows] = tb["x"]
    ta["slot"].fill_(-1)
    for k, c in (("pos", rows), ("slot", rows), ("idx", nnz), ("kv_pos", nnz)):
        ta[k][:c] = tb[k][:c]
    ta["k"].copy_(akv.to_device(b.k, "bf16"))
    ta["v"].copy_(akv.to_device(b.v, "bf16"))
    for k in ("q_ptr", "kv_ptr", "keep", "qw", "kw"):
        ta[k].copy_(tb[k])
    g.replay()
    torch.cuda.synchronize()
    kept = int(tb["o_ptr"][-1])
    for k, c in (("q", rows), ("out", rows), ("lse", rows), ("mass", 3), ("o_ptr", 4), ("o_idx", kept),
                 ("o_pos", kept), ("d_ptr", 4)):
        assert torch.equal(ta[k][:c], tb[k][:c]), k


def test_two_streams_at_once():
    """Two batches on two streams, each with its own workspace, enqueued in
    turn many times: the results of each alone."""
    torch = _torch()
    bts = [Batch(41, [1, 1, 1], [3000, 900, 33], 16, 4, "bf16"),
           Batch(42, [40, 9, 70], [800, 900, 333], 16, 4, "bf16")]
    ts = [_step_tensors(b, 43) for b in bts]
    masses = [t["mass"].clone() for t in ts]
    alone = []
    for b, t, m in zip(bts, ts, masses):
        _step(b, t)
        torch.cuda.synchronize()
        alone.append({k: t[k].clone() for k in ("out", "lse", "mass", "o_idx")})
    streams = [torch.cuda.Stream() for _ in bts]
    for _ in range(10):
        for b, t, m, s in zip(bts, ts, masses, streams):
            with torch.cuda.stream(s):
                t["mass"].copy_(m)
                _step(b, t)
    torch.cuda.synchronize()
    for t, want in zip(ts, alone):
        for k, w in want.items():
            assert torch.equal(t[k], w), k


def test_binding_refuses_wrong_tensors():
    torch = _torch()
    bt = Batch(51, [2], [40], 16, 4, "bf16")
    d = bt.device()
    out, lse = run_chunk(bt, d)
    for k, bad in (("idx", d["idx"].long()), ("q_ptr", d["q_ptr"].cpu()), ("q", d["q"].float()),
                   ("kv_ptr", d["kv_ptr"][:1]), ("v", d["v"][:, :, :32].contiguous())):
        with pytest.raises(ValueError):
            run_chunk(bt, {**d, k: bad})
    with pytest.raises(ValueError):
        run_mass(bt, d, lse, None, 1.0, torch.zeros(2, 40, device="cuda"))
    x = torch.zeros(2, 24, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):  # heads of a token not contiguous
        akv.akv_qk_norm_append(bt.shp, 2, x[:, :16].transpose(0, 1).contiguous().transpose(0, 1),
                               x[:, 16:20].contiguous(), x[:, 20:].contiguous(), akv.i32_device([0, 1]),
                               akv.i32_device([0, 1]), d["k"], d["v"], torch.empty_like(d["q"]))
