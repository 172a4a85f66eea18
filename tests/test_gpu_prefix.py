"""Attention of a batch whose requests share prefixes, against its definition in
64 bits (tests/_kv8.py; the tolerances are those of the chunk calls), and the 8-bit
cache and the shared prefix run together as a serving step does."""
import numpy as np
import pytest

import kv_cache_drop_gb300 as akv
import oracle
import workloads
from _kv8 import attend, decode, held, quantise, turn

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _rand(rng, shape, dtype, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return workloads.bf16_bits(x) if dtype == "bf16" else x


class Batch:
    """Requests of m[b] rows over own lists of n[b] entries; groups of
    consecutive requests (`cut`: their first requests, then the end) over prefixes
    of p[g] entries; `lead` rows before the first group's and the first request's."""

    def __init__(self, seed, m, n, cut, p, Hq, Hkv, dtype, scale=1.0, lead=0, tail=2):
        rng = np.random.default_rng(seed)
        self.m, self.n, self.p, self.Hq, self.Hkv, self.dtype = m, n, p, Hq, Hkv, dtype
        ptr = lambda x, o=0: (o + np.concatenate([[0], np.cumsum(x)])).astype(np.int32)  # noqa: E731
        self.q_ptr, self.kv_ptr, self.pre_ptr = ptr(m, lead), ptr(n), ptr(p)
        self.g_ptr = self.q_ptr[cut].astype(np.int32)
        self.B, self.G, self.rows = len(m), len(p), int(self.q_ptr[-1]) + tail
        nn, pp = int(self.kv_ptr[-1]), int(self.pre_ptr[-1])
        self.S = nn + pp + 5
        free = rng.permutation(self.S).astype(np.int32)
        self.idx, self.pre = free[:nn].copy(), free[nn:nn + pp].copy()
        self.q = _rand(rng, (self.rows, Hq, 64), dtype, scale)
        self.k, self.v = (_rand(rng, (self.S, Hkv, 64), dtype) for _ in range(2))
        self.shp = akv.shape(Hq, Hkv, 64, dtype)
        self.sizes = dict(max_rows=int(np.diff(self.g_ptr).max(initial=0)), max_prefix=max(p, default=0),
                          max_q=max(m, default=0), max_kv=max(n, default=0))

    def device(self):
        return dict(q=akv.to_device(self.q, self.dtype), k=akv.to_device(self.k, self.dtype),
                    v=akv.to_device(self.v, self.dtype),
                    **{x: akv.i32_device(getattr(self, x)) for x in ("q_ptr", "kv_ptr", "pre_ptr", "g_ptr",
                                                                     "idx", "pre")})

    def workspace(self, **sizes):
        torch = _torch()
        sizes = {**self.sizes, **sizes}
        return torch.full((akv.akv_prefix_workspace(self.shp, self.G, self.B, self.rows, **sizes),), 255,
                          dtype=torch.uint8, device="cuda")

    def run(self, d, lse=True, out=None, l=None, ws=None, stream=None, **sizes):  # noqa: E741
        torch = _torch()
        out = torch.full_like(d["q"], 7.0) if out is None else out
        if l is None and lse:
            l = torch.full((self.rows, self.Hq), 7.0, device="cuda")  # noqa: E741
        ws = self.workspace(**sizes) if ws is None else ws
        akv.akv_prefix_attention(self.shp, self.G, d["g_ptr"], d["pre_ptr"], d["pre"], self.B, d["q_ptr"],
                                 d["q"], d["k"], d["v"], d["kv_ptr"], d["idx"], out=out, lse=l, workspace=ws,
                                 stream=stream, **{**self.sizes, **sizes})
        assert akv.akv_workspace_status(ws, stream=stream) == 0
        return out, l

    def want(self, t):
        """(out, lse, tolerances) of row t [1, Hq, ...], None where no list is its."""
        wide = lambda x: oracle.widen(x, self.dtype).astype(np.float64)  # noqa: E731
        parts = []
        for g in range(self.G):
            if self.g_ptr[g] <= t < self.g_ptr[g + 1]:
                at = self.pre[self.pre_ptr[g]:self.pre_ptr[g + 1]]
                parts.append((wide(self.k[at]), wide(self.v[at]), [self.p[g]]))
        for b in range(self.B):
            if self.q_ptr[b] <= t < self.q_ptr[b + 1]:
                at = self.idx[self.kv_ptr[b]:self.kv_ptr[b + 1]]
                i = t - self.q_ptr[b]
                parts.append((wide(self.k[at]), wide(self.v[at]), [max(0, self.n[b] - self.m[b] + 1 + i)]))
        return attend(wide(self.q[t:t + 1]), parts, self.dtype) if parts else None

    def check(self, out, lse, rows=None, fill=7.0):
        o = out.float().cpu().numpy().astype(np.float64)
        g = None if lse is None else lse.cpu().numpy().astype(np.float64)
        for t in range(self.rows) if rows is None else rows:
            w = self.want(t)
            if w is None:
                assert np.all(o[t] == fill) and (g is None or np.all(g[t] == fill)), t
                continue
            err = np.abs(o[t] - w[0][0])
            assert np.all(err <= w[2][0]), (t, float((err / np.maximum(w[2][0], 1e-300)).max()))
            if g is not None:
                none = np.isneginf(w[1][0])
                assert np.array_equal(np.isneginf(g[t]), none)
                assert np.all(np.abs(g[t][~none] - w[1][0][~none]) <= w[3][0][~none]), t


# name: rows, own lists, groups' first requests, prefixes
SHAPES = {
    "one group of single tokens": ([1] * 5, [1, 2, 129, 700, 33], [0, 5], [515]),
    "empty lists": ([1, 2, 0, 3, 1], [0, 1, 5, 0, 9], [0, 2, 5], [0, 65]),
    "tile edges": ([15, 17, 16, 33, 1], [96, 97, 16, 200, 95], [0, 1, 3, 5], [96, 191, 1]),
    "chunks": ([70, 1, 130, 5], [300, 1, 131, 500], [0, 3, 4], [193, 2000]),
    "short prefix, long lists": ([1, 1], [9000, 4000], [0, 2], [1]),
    "long prefix": ([1, 1, 2], [3, 1, 40], [0, 3], [9001]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 4), (24, 3), (2, 2), (20, 1)])
@pytest.mark.parametrize("name", list(SHAPES))
def test_prefix_attention(name, Hq, Hkv, dtype):
    torch = _torch()
    m, n, cut, p = SHAPES[name]
    bt = Batch(len(name) + Hq, m, n, cut, p, Hq, Hkv, dtype, lead=3)
    d = bt.device()
    out, lse = bt.run(d)
    bt.check(out, lse)
    again, l2 = bt.run(d)
    assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups_and_requests_that_cover_other_rows(dtype):
    """Rows in a group and no request, in a request and no group, in neither; a
    group's limit inside a request; no groups; no requests; lse left out."""
    torch = _torch()
    bt = Batch(5, [6, 40, 3], [10, 90, 2], [0, 3], [130], 16, 4, dtype, lead=4, tail=20)
    bt.g_ptr = np.array([1, 30], np.int32)  # inside the second request
    bt.sizes["max_rows"] = 29
    d = bt.device()
    bt.check(*bt.run(d))
    bt.g_ptr = np.array([20, bt.rows - 3], np.int32)
    bt.sizes["max_rows"] = bt.rows
    d = bt.device()
    bt.check(*bt.run(d))
    bt.check(bt.run(d, lse=False)[0], None)
    # no requests
    q_ptr, B = bt.q_ptr, bt.B
    bt.B, bt.sizes["max_q"], bt.sizes["max_kv"] = 0, 0, 0
    d["q_ptr"] = d["kv_ptr"] = akv.i32_device([0])
    bt.check(*bt.run(d))
    # no groups: as akv_chunk_attention
    bt = Batch(6, [6, 40, 3], [10, 90, 2], [0], [], 16, 4, dtype)
    d = bt.device()
    out, lse = bt.run(d)
    bt.check(out, lse)
    o2, l2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    ws = torch.empty(akv.akv_chunk_workspace(bt.shp, bt.B, bt.rows, 40, 90), dtype=torch.uint8, device="cuda")
    akv.akv_chunk_attention(bt.shp, bt.B, d["q_ptr"], d["q"], d["k"], d["v"], d["kv_ptr"], d["idx"], 40, 90, o2,
                            l2, ws)
    err = (out.float() - o2.float()).abs().max().item()
    assert err <= (2.0 ** -6 if dtype == "bf16" else 2.0 ** -18)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 9, 40, 150])
def test_nothing_anywhere(rows, dtype):
    """Empty lists: zeros and -inf, with bounds of 0 and with larger ones."""
    for bound in (0, 700):
        bt = Batch(7, [rows, rows], [0, 0], [0, 2], [0], 16, 4, dtype)
        d = bt.device()
        out, lse = bt.run(d, max_prefix=bound, max_kv=bound)
        bt.check(out, lse)
        assert not out[:2 * rows].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 10, 40])
def test_hidden_values_and_jumping_scores(m, dtype):
    """Own entries that a row does not see hold infinities and NaN; scores of
    standard deviation 16, so that one list or the other carries a row."""
    torch = _torch()
    bt = Batch(8, [m, m], [1500, 333], [0, 2], [700], 16, 4, dtype, scale=16)
    d = bt.device()
    if m > 1:  # the last row's entry is hidden from the others
        for b in range(2):
            at = int(bt.idx[bt.kv_ptr[b + 1] - 1])
            d["v"][at, 0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
            bt.v[at, 0, :3] = 0
    out, lse = bt.run(d)
    last = {int(bt.q_ptr[1]) - 1, int(bt.q_ptr[2]) - 1} if m > 1 else set()
    bt.check(out, lse, [t for t in range(bt.rows) if t not in last])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_cut_the_lists(dtype):
    """Entries past max_prefix and max_kv have no part; larger bounds change nothing."""
    bt = Batch(9, [1, 3], [50, 90], [0, 2], [300], 16, 4, dtype)
    d = bt.device()
    bt.check(*bt.run(d, max_prefix=5000, max_kv=4000, max_q=60, max_rows=300))
    out, lse = bt.run(d, max_prefix=100, max_kv=50)
    cut = Batch(9, [1, 3], [50, 90], [0, 2], [300], 16, 4, dtype)
    cut.p, cut.n = [100], [50, 50]
    cut.pre = cut.pre[:100]
    cut.pre_ptr = np.array([0, 100], np.int32)
    cut.idx = np.concatenate([cut.idx[:50], cut.idx[50:100]])
    cut.kv_ptr = np.array([0, 50, 100], np.int32)
    cut.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_on_two_streams(dtype):
    torch = _torch()
    a = Batch(10, [1, 5, 2], [300, 77, 2], [0, 2, 3], [400, 9], 24, 3, dtype)
    b = Batch(11, [5, 1, 2], [5, 300, 74], [0, 1, 3], [9, 400], 24, 3, dtype)
    sizes = dict(max_rows=8, max_prefix=400, max_q=5, max_kv=300)
    d, e = a.device(), b.device()
    out, lse = torch.full_like(d["q"], 7.0), torch.full((a.rows, 24), 7.0, device="cuda")
    ws = a.workspace(**sizes)
    a.run(d, out=out, l=lse, ws=ws, **sizes)
    g = torch.cuda.CUDAGraph()
    args = (a.shp, a.G, d["g_ptr"], d["pre_ptr"], d["pre"], a.B, d["q_ptr"], d["q"], d["k"], d["v"], d["kv_ptr"],
            d["idx"])
    with torch.cuda.graph(g):
        akv.akv_prefix_attention(*args, out=out, lse=lse, workspace=ws, **sizes)
    g.replay()
    a.check(out, lse)
    for k, x in e.items():
        if d[k].shape[0] >= x.shape[0]:
            d[k][:x.shape[0]].copy_(x)
        else:
            pytest.fail("the second batch is larger")
    g.replay()
    b.check(out, lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    bts = [Batch(12 + i, [1, 40 + i], [900, 700], [0, 2], [2000], 16, 4, dtype) for i in range(2)]
    ds, wss = [x.device() for x in bts], [x.workspace() for x in bts]
    outs = [torch.full_like(x["q"], 7.0) for x in ds]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(streams):
            x, y = bts[i], ds[i]
            akv.akv_prefix_attention(x.shp, x.G, y["g_ptr"], y["pre_ptr"], y["pre"], x.B, y["q_ptr"], y["q"],
                                     y["k"], y["v"], y["kv_ptr"], y["idx"], out=outs[i], lse=None,
                                     workspace=wss[i], stream=s, **x.sizes)
    torch.cuda.synchronize()
    for x, o in zip(bts, outs):
        x.check(o, None)


def test_many_requests_of_one_group():
    """300 requests behind one prefix: several row tiles of one group."""
    rng = np.random.default_rng(3)
    m = [0 if b % 7 == 3 else 1 for b in range(300)]
    n = [int(rng.integers(0, 60)) for _ in range(300)]
    bt = Batch(13, m, n, [0, 300], [777], 16, 4, "bf16")
    bt.check(*bt.run(bt.device()))


def test_a_fleet_over_an_8_bit_prefix():
    """Written in 8 bits, decoded there, read back into a bf16 pool and attended
    over once for all requests; the mass of the own entries from the joint lse."""
    torch = _torch()
    rng = np.random.default_rng(21)
    Hq, Hkv, P, B = 16, 4, 600, 6
    shp = akv.shape(Hq, Hkv)
    own = [40, 1, 77, 16, 5, 130]
    ptr = np.concatenate([[0], np.cumsum(own)]).astype(np.int32)
    # the prompt's raw rows, written into an 8-bit pool
    k, v = (_rand(rng, (P, Hkv, 64), "bf16") for _ in range(2))
    S8 = P + 9
    slot = rng.permutation(S8)[:P].astype(np.int32)
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    pool = [torch.zeros(S8, Hkv, 64, dtype=torch.uint8, device="cuda").view(f8) for _ in range(2)]
    scale = [torch.zeros(S8, Hkv, dtype=torch.uint8, device="cuda").view(e8) for _ in range(2)]
    akv.akv_append_kv_q8(shp, P, akv.to_device(k, "bf16"), akv.to_device(v, "bf16"), akv.i32_device(slot), *pool,
                         *scale)
    K8, V8 = (held(*quantise(oracle.widen(x, "bf16"))) for x in (k, v))
    # one request decodes over it there
    q1 = _rand(rng, (1, Hq, 64), "bf16")
    out1 = torch.zeros(1, Hq, 64, dtype=torch.bfloat16, device="cuda")
    ws1 = torch.empty(akv.akv_decode_q8_workspace(shp, 1, P), dtype=torch.uint8, device="cuda")
    akv.akv_decode_attention_q8(shp, 1, akv.to_device(q1, "bf16"), akv.i32_device([P]), None, None, None, *pool,
                                *scale, akv.i32_device([0, P]), akv.i32_device(slot),
                                akv.i32_device(np.arange(P)), P, out1, ws1)
    want, tol = decode(oracle.widen(q1, "bf16")[0].astype(np.float64), P, K8, V8, np.arange(P), "bf16")
    assert np.all(np.abs(out1[0].float().cpu().numpy() - want) <= tol)
    # a group runs: its prefix back in the bf16 pool, rotated, behind the own entries
    S = int(ptr[-1]) + P + 3
    kp, vp = (_rand(rng, (S, Hkv, 64), "bf16") for _ in range(2))
    free = rng.permutation(S).astype(np.int32)
    idx, pre = free[:ptr[-1]].copy(), free[ptr[-1]:ptr[-1] + P].copy()
    kd, vd = akv.to_device(kp, "bf16"), akv.to_device(vp, "bf16")
    akv.akv_read_kv_q8(shp, P, akv.i32_device(slot), akv.i32_device(np.arange(P)), akv.i32_device(pre), *pool,
                       *scale, kd, vd)
    q = _rand(rng, (B, Hq, 64), "bf16")
    qd = akv.to_device(q, "bf16")
    out, lse = torch.zeros_like(qd), torch.zeros(B, Hq, device="cuda")
    sizes = dict(max_rows=B, max_prefix=P, max_q=1, max_kv=max(own))
    ws = torch.empty(akv.akv_prefix_workspace(shp, 1, B, B, **sizes), dtype=torch.uint8, device="cuda")
    rows = akv.i32_device(np.arange(B + 1))
    akv.akv_prefix_attention(shp, 1, akv.i32_device([0, B]), akv.i32_device([0, P]), akv.i32_device(pre), B, rows,
                             qd, kd, vd, akv.i32_device(ptr), akv.i32_device(idx), out=out, lse=lse, workspace=ws,
                             **sizes)
    mass = torch.zeros(B, max(own), device="cuda")
    wm = torch.empty(akv.akv_attention_mass_workspace(shp, B, B, 1, max(own)), dtype=torch.uint8, device="cuda")
    akv.akv_attention_mass(shp, B, rows, qd, kd, akv.i32_device(ptr), akv.i32_device(idx), 1, max(own), lse, 1.0,
                           None, mass, wm)
    Kp, Vp = oracle.widen(kp, "bf16").astype(np.float64), oracle.widen(vp, "bf16").astype(np.float64)
    Kr = turn(K8, np.arange(P))
    bf = lambda x: oracle.widen(workloads.bf16_bits(x.astype(np.float32)), "bf16").astype(np.float64)  # noqa: E731
    got, ql = out.float().cpu().numpy(), oracle.widen(q, "bf16").astype(np.float64)
    for b in range(B):
        at = idx[ptr[b]:ptr[b + 1]]
        w, l64, tol, tl = attend(ql[b:b + 1], [(bf(Kr), V8, [P]), (Kp[at], Vp[at], [own[b]])], "bf16")
        # a key read back is rounded from a value 2^-20 of its pair off: it may go
        # to the neighbouring bf16 number, 2^-7 of itself, here and there
        E = 2.0 ** -7 * np.einsum("hd,jhd->hj", np.abs(ql[b]), np.abs(np.repeat(Kr, 4, 1))).max(-1) / 8
        assert np.all(np.abs(got[b] - w[0]) <= tol[0] + np.expm1(2 * E)[:, None] * np.abs(V8).max())
        s = np.einsum("hd,jhd->hj", ql[b], np.repeat(Kp[at], 4, 1)) / 8
        m64 = np.exp(s - lse[b].cpu().numpy()[:, None]).sum(0)
        assert np.allclose(mass[b, :own[b]].cpu().numpy(), m64, rtol=2.0 ** -12)
