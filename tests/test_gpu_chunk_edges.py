"""Edges of the calls over a chunk of new tokens: what their definitions allow
and ordinary batches do not reach.  Batches, references and tolerances are
those of test_gpu_chunk.py."""
import copy
import math

import numpy as np
import pytest

import kv_cache_drop_gb300 as akv
import oracle
import workloads
from test_gpu_chunk import (Batch, _close_rows, _evict_ref, _host, _prepared, _rand, _torch, check_chunk,
                            check_mass, run_chunk, run_mass)

pytestmark = pytest.mark.gpu


def _levels(bt, level, seed):
    """Every row's scores are 32 level[j], the values N(0, 1)."""
    rng = np.random.default_rng(seed)
    k, v = np.zeros((bt.S, bt.Hkv, 64), np.float32), np.zeros((bt.S, bt.Hkv, 64), np.float32)
    for b in range(bt.B):
        at, n = bt.idx[bt.kv_ptr[b]:bt.kv_ptr[b + 1]], bt.n[b]
        k[at] = level[:n, None, None]
        v[at] = rng.standard_normal((n, bt.Hkv, 64))
    put = workloads.bf16_bits if bt.dtype == "bf16" else lambda x: x
    bt.q = put(np.full((bt.rows, bt.Hq, 64), 4, np.float32))
    bt.k, bt.v = put(k), put(v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 10, 40, 300])
@pytest.mark.parametrize("case", ["one", "some", "rising", "then low"])
def test_chunk_large_values(case, m, dtype):
    """Values of 2^48 to 2^100 under scores that jump by up to 54 (2^78) after
    entries without any: the output is an average of values, so it is finite,
    and it and its tolerance scale with them."""
    n = 1500
    j = np.arange(n)
    level = {"one": np.where(j == 700, 1.25, 0), "some": np.where(j % 250 == 200, 1.6875, 0),
             "rising": np.minimum(j // 100, 12) * 0.140625,  # by 4.5 at a time, 54 in all
             "then low": np.where(j < 300, 0, np.where(j < 400, 1.6875, -2))}[case]
    want = None
    for B in (1, 20):  # lists in splits, and (more than 16 rows) whole
        bt = Batch(60, [m] * B, [n] * B, 16, 4, dtype)
        _levels(bt, level, 61)
        want = want or bt.attend(0)  # request 0 is the same in both
        d = bt.device()
        v = d["v"]
        for power in (0, 48, 60, 72, 100):
            d["v"] = v * 2.0 ** power
            out, lse = run_chunk(bt, d)
            assert bool(_torch().isfinite(out.float()).all()), power
            o, l = _host(out)[:m] / 2.0 ** power, _host(lse)[:m]
            assert np.all(np.abs(o - want[0]) <= want[2]), power
            assert np.all(np.abs(l - want[1]) <= want[3]), power


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 40, 300])
def test_chunk_infinite_value_seen_by_all(m, dtype):
    """An infinity among the first entries' values is every row's output in
    its column, and no other's."""
    bt = Batch(62, [m], [1500], 16, 4, dtype)
    d = bt.device()
    at = int(bt.idx[5])
    d["v"][at, 1, 9] = float("inf")
    d["v"][at, 2, 11] = -float("inf")
    out, lse = run_chunk(bt, d)
    o = _host(out)
    assert np.all(o[:, 4:8, 9] == np.inf) and np.all(o[:, 8:12, 11] == -np.inf)
    want, _, tol, _ = bt.attend(0)
    rest = np.ones(o.shape, bool)
    rest[:, 4:8, 9] = rest[:, 8:12, 11] = False
    assert np.all((np.abs(o - want) <= tol)[rest])


@pytest.mark.parametrize("lens", [[1], [700, 0, 33], [20000, 5]])
def test_evict_exactly_sized_outputs(lens):
    """Buffers of exactly the kept and dropped entries, the empty ones among
    them (an empty tensor has no address)."""
    torch = _torch()
    rng = np.random.default_rng(67)
    B, ptr = len(lens), np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    nnz, wide = int(ptr[-1]), max(lens)
    idx, pos = (rng.permutation(nnz).astype(np.int32) for _ in range(2))
    mass = rng.random((B, wide)).astype(np.float32)
    i32 = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
    for keep in (0, wide, wide // 3):
        for with_pos in (True, False):
            kept = [_evict_ref(mass[b], n, keep, 1, 1) for b, n in enumerate(lens)]
            n_kept, width = sum(map(len, kept)), max(map(len, kept))
            o_ptr, o_idx, d_ptr, drop = i32(B + 1), i32(n_kept), i32(B + 1), i32(nnz - n_kept)
            o_pos = i32(n_kept) if with_pos else None
            o_mass = torch.full((B, width), -9.0, device="cuda")
            akv.akv_evict_by_mass(B, akv.i32_device(ptr), akv.i32_device(idx),
                                  akv.i32_device(pos) if with_pos else None, wide,
                                  torch.from_numpy(mass).cuda(), akv.i32_device([keep] * B), 1, 1, o_ptr,
                                  o_idx, o_pos, o_mass, d_ptr, drop)
            torch.cuda.synchronize()
            at = np.concatenate([ptr[b] + k for b, k in enumerate(kept)]).astype(np.int64)
            gone = np.concatenate([ptr[b] + np.setdiff1d(np.arange(lens[b]), k) for b, k in enumerate(kept)])
            np.testing.assert_array_equal(o_idx.cpu().numpy(), idx[at])
            np.testing.assert_array_equal(drop.cpu().numpy(), idx[gone.astype(np.int64)])
            if with_pos:
                np.testing.assert_array_equal(o_pos.cpu().numpy(), pos[at])
            for b, k in enumerate(kept):
                np.testing.assert_array_equal(o_mass[b, :len(k)].cpu().numpy(), mass[b, k])
            assert o_ptr.tolist() == np.concatenate([[0], np.cumsum([len(k) for k in kept])]).tolist()
            assert int(d_ptr[-1]) == nnz - n_kept


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 10, 40, 300])
@pytest.mark.parametrize("S", [0, 5])
def test_lists_without_entries_under_a_bound(S, m, dtype):
    """kv_indices of no entries while max_kv allows some: rows see nothing,
    nothing gains mass, nothing is kept or dropped."""
    torch = _torch()
    shp = akv.shape(16, 4, 64, dtype)
    q = akv.to_device(_rand(np.random.default_rng(1), (2 * m, 16, 64), dtype), dtype)
    pool, ptr, none = q.new_zeros(S, 4, 64), akv.i32_device([0, 0, 0]), akv.i32_device([])
    qp = akv.i32_device([0, m, 2 * m])
    out, lse = torch.full_like(q, 7.0), torch.zeros(2 * m, 16, device="cuda")
    ws = torch.empty(akv.akv_chunk_workspace(shp, 2, 2 * m, m, 5000), dtype=torch.uint8, device="cuda")
    akv.akv_chunk_attention(shp, 2, qp, q, pool, pool, ptr, none, m, 5000, out, lse, ws)
    torch.cuda.synchronize()
    assert not out.any() and bool(torch.isneginf(lse).all())
    ws = torch.empty(akv.akv_attention_mass_workspace(shp, 2, 2 * m, m, 5000), dtype=torch.uint8,
                     device="cuda")
    mass = torch.full((2, 5000), -3.0, device="cuda")
    akv.akv_attention_mass(shp, 2, qp, q, pool, ptr, none, m, 5000, lse, 0.5, mass, mass, ws)
    o_ptr, d_ptr = (torch.full((3,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    akv.akv_evict_by_mass(2, ptr, none, none, 5000, mass, akv.i32_device([10, 0]), 1, 1, o_ptr, none, none,
                          mass.clone(), d_ptr, none)
    torch.cuda.synchronize()
    assert bool((mass == -3).all()) and not o_ptr.any() and not d_ptr.any()


def test_append_to_a_pool_without_slots():
    """S = 0: every token is padding."""
    torch = _torch()
    shp = akv.shape(16, 4, 64, "bf16")
    x = torch.ones(3, 24, 64, dtype=torch.bfloat16, device="cuda")
    pool, qo = x.new_zeros(0, 4, 64), torch.full((3, 16, 64), 7.0, dtype=x.dtype, device="cuda")
    akv.akv_qk_norm_append(shp, 3, x[:, :16], x[:, 16:20], x[:, 20:], akv.i32_device([0, 1, 2]),
                           akv.i32_device([0, -1, 5]), pool, pool, qo)
    torch.cuda.synchronize()
    assert bool((qo == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [4, 6, 12, 40])
def test_mass_has_no_bias(m, dtype):
    """Weights exp(L - L) = 1 for some 120 values of L between 45 and 88, with
    q . k exact (one product): each is off by the rounding of L's product with
    log2 e, half a step of [64, 128) either way, which averages out.  Mean of
    N = 121 roundings, uniform over a step of 2^-17, times ln 2: a standard
    deviation of 1.4e-7; four of these, and 2^-22 for the exponential, are
    8e-7."""
    torch = _torch()
    L = np.concatenate([np.arange(45, 64, 0.25), np.arange(64, 86.5, 0.5)])
    B, n = len(L), m + 260
    bt = Batch(63, [m] * B, [n] * B, 16, 4, dtype)
    q, k = np.zeros((bt.rows, 16, 64), np.float32), np.zeros((bt.S, 4, 64), np.float32)
    q[..., 0] = 8
    for b in range(B):
        k[bt.idx[bt.kv_ptr[b]:bt.kv_ptr[b + 1]], :, 0] = L[b]
    bt.q, bt.k = (workloads.bf16_bits(x) if dtype == "bf16" else x for x in (q, k))
    d = bt.device()
    lse = torch.from_numpy(np.repeat(L, m).astype(np.float32)).cuda()[:, None].repeat(1, 16)
    got = torch.zeros(B, n, device="cuda")
    run_mass(bt, d, lse, None, 1.0, got)
    check_mass(bt, lse, None, 1.0, got, 0.0)
    w = _host(got)[:, :256] / (16 * m)  # entries that every row sees
    assert abs(w.mean() - 1) < 8e-7, w.mean() - 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 6, 14, 40, 300])
def test_mass_of_an_exact_lse(m, dtype):
    """A log-sum-exp that is not the library's own but the definition's,
    rounded to fp32."""
    torch = _torch()
    bt = Batch(64, [m, m], [900, m + 1], 16, 4, dtype, scale=3.0)
    d = bt.device()
    lse = torch.from_numpy(np.concatenate([bt.attend(b)[1] for b in range(2)]).astype(np.float32)).cuda()
    got = torch.zeros(2, 900, device="cuda")
    run_mass(bt, d, lse, None, 1.0, got)
    check_mass(bt, lse, None, 1.0, got, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [2, 6, 14, 40, 300])
def test_mass_rows_that_count_nothing(m, dtype):
    """Rows whose log-sum-exp is -inf count nothing, whatever they hold: NaN,
    infinities, zeros."""
    torch = _torch()
    bt = Batch(65, [m, m], [900, m + 70], 16, 4, dtype)
    d = bt.device()
    _, lse = run_chunk(bt, d)
    out_rows = np.arange(0, 2 * m, 2)
    at = torch.from_numpy(out_rows).cuda()
    lse[at] = -math.inf
    want = torch.zeros(2, 900, device="cuda")
    run_mass(bt, d, lse, None, 1.0, want)
    check_mass(bt, lse, None, 1.0, want, 0.0)
    for bad in (math.nan, math.inf, -math.inf, 0.0):
        d["q"][at] = bad
        got = torch.zeros(2, 900, device="cuda")
        run_mass(bt, d, lse, None, 1.0, got)
        assert torch.equal(got, want), bad


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
def test_qk_norm_of_any_magnitude(n, dtype):
    """Rows over the range whose squares fp32 holds: up to 2^60, and down to
    2^-55 or, beside an eps, to anything."""
    torch = _torch()
    rng = np.random.default_rng(66)
    Hq, Hkv = 16, 4
    shp = akv.shape(Hq, Hkv, 64, dtype)
    x = rng.standard_normal((n, Hq + 2 * Hkv, 64)).clip(-3, 3)
    for eps, powers in ((0.0, [-53, -20, 0, 20, 58]), (1e-30, [-100, -55, -20, 0, 58]),
                        (1e-6, [-120, -50, -20, -8, 0, 58])):
        p = np.resize(np.array(powers), n * (Hq + 2 * Hkv)).reshape(n, -1, 1)
        y = (x * 2.0 ** p).astype(np.float32)
        y = workloads.bf16_bits(y) if dtype == "bf16" else y
        pos = rng.integers(0, 1000, size=n).astype(np.int32)
        t = akv.to_device(y, dtype)
        kp, vp = (torch.zeros(n, Hkv, 64, dtype=t.dtype, device="cuda") for _ in range(2))
        qo = torch.zeros(n, Hq, 64, dtype=t.dtype, device="cuda")
        akv.akv_qk_norm_append(shp, n, t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], akv.i32_device(pos),
                               akv.i32_device(np.arange(n)), kp, vp, qo, eps=eps)
        torch.cuda.synchronize()
        _close_rows(_host(qo), _prepared(y[:, :Hq], None, pos, 1, 1, eps, dtype), dtype)
        _close_rows(_host(kp), _prepared(y[:, Hq:Hq + Hkv], None, pos, 1, 1, eps, dtype), dtype)
        assert np.array_equal(_host(vp), oracle.widen(y[:, Hq + Hkv:], dtype))


class Led(Batch):
    """A batch whose rows come after `lead` rows of q that belong to no
    request."""

    def __init__(self, *args, lead=0, tail=0, **kw):
        super().__init__(*args, tail=lead + tail, **kw)
        self.lead = lead
        self.q_ptr = self.q_ptr + np.int32(lead)


def _cut(bt, max_q, max_kv):
    """The batch that a call with these bounds sees: each chunk's first max_q
    rows over its list's first max_kv entries."""
    c = copy.copy(bt)
    c.m, c.n = [min(x, max_q) for x in bt.m], [min(x, max_kv) for x in bt.n]
    c.q = np.concatenate([bt.q[p:p + x] for p, x in zip(bt.q_ptr, c.m)])
    c.idx = np.concatenate([bt.idx[p:p + x] for p, x in zip(bt.kv_ptr, c.n)])
    c.q_ptr = np.concatenate([[0], np.cumsum(c.m)]).astype(np.int32)
    c.kv_ptr = np.concatenate([[0], np.cumsum(c.n)]).astype(np.int32)
    c.rows = int(c.q_ptr[-1])
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [([2, 0, 3], [5000, 10, 70]), ([10, 6, 0, 16], [3000, 3100, 8, 40]),
                                 ([30, 20], [5000, 900]), ([100, 1, 51], [2500, 3000, 60])])
def test_chunk_rows_and_bounds(m, n, dtype):
    """Rows before the first request and after the last, and chunks and lists
    longer than max_q and max_kv: cut to them, with every row and entry past
    the cut left as it was."""
    torch = _torch()
    bt = Led(68, m, n, 16, 4, dtype, lead=5, tail=4)
    d = bt.device()
    mq, mk = max(m), max(n)
    for max_q, max_kv in ((mq, mk), (mq + 9, mk + 900), (mq - 1, mk), (mq, mk - 7), ((mq + 1) // 2, mk // 2)):
        c = _cut(bt, max_q, max_kv)
        out, lse = run_chunk(bt, d, max_q=max_q, max_kv=max_kv)
        torch.cuda.synchronize()
        mine = np.concatenate([np.arange(p, p + x) for p, x in zip(bt.q_ptr, c.m)])
        rest = np.setdiff1d(np.arange(bt.rows), mine)
        at = torch.from_numpy(mine).cuda()
        check_chunk(c, out[at], lse[at])
        assert np.all(_host(out)[rest] == 7) and np.all(_host(lse)[rest] == 7)
        mass_in = torch.rand(bt.B, mk + 900, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
        got = torch.full((bt.B, mk + 900), -3.0, device="cuda")
        run_mass(bt, d, lse, mass_in, 0.5, got, max_q=max_q, max_kv=max_kv)
        check_mass(c, lse[at], mass_in, 0.5, got, -3.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_chunk_among_single_tokens(dtype):
    """A prefill chunk batched with decode steps: 13 single tokens and 260
    rows over lists of 1 to 4,000 entries."""
    torch = _torch()
    rng = np.random.default_rng(69)
    m = [1] * 6 + [260] + [1] * 7
    n = [int(x) for x in rng.integers(1, 4000, size=14)]
    n[6], n[0], n[13] = 1300, 4000, 1
    bt = Batch(70, m, n, 16, 4, dtype)
    d = bt.device()
    out, lse = run_chunk(bt, d)
    check_chunk(bt, out, lse)
    got = torch.zeros(bt.B, bt.max_kv, device="cuda")
    run_mass(bt, d, lse, None, 1.0, got)
    check_mass(bt, lse, None, 1.0, got, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 6, 14, 40, 300])
@pytest.mark.parametrize("scale", [0.0, 1.0, 6.0])
def test_mass_of_the_library_lse_sums_to_the_rows(scale, m, dtype):
    """Attention's log-sum-exp into the mass: every row and head gives a mass
    of 1.  Off by the lse's error and the weights': 2^-22 (1 + |lse|) for the
    roundings of lse and of its products with ln 2 and log2 e, and nine steps of
    a tensor core that cuts each sum (four in the attention, five in the mass),
    each below 2^-23 of the sum of the products' sizes."""
    torch = _torch()
    bt = Batch(71, [m, m], [1200, m + 5], 16, 4, dtype, scale=scale)
    d = bt.device()
    _, lse = run_chunk(bt, d)
    got = torch.zeros(2, 1200, device="cuda")
    run_mass(bt, d, lse, None, 1.0, got)
    total, l = _host(got).sum(1), np.abs(_host(lse))
    for b in range(2):
        _, E = bt.scores(b)  # 2^-18 of that size
        tol = 2.0 ** -22 * (1 + l[bt.q_ptr[b]:bt.q_ptr[b + 1]].max()) + 9 * 2.0 ** -5 * E.max()
        assert abs(total[b] / (16 * m) - 1) <= tol, (total[b] / (16 * m) - 1, tol)
