"""The 8-bit cache: rows written (bit for bit), read back, and decoded with
rotation on read, against their definitions in 64 bits (tests/_kv8.py derives the
tolerances)."""
import numpy as np
import pytest

import kv_cache_drop_gb300 as akv
import oracle
import workloads
from _kv8 import VALUES, decode, held, quantise, turn

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _bits(x, dtype):
    return workloads.bf16_bits(x.astype(np.float32)) if dtype == "bf16" else x.astype(np.float32)


def _wide(x, dtype):
    return oracle.widen(x, dtype).astype(np.float64)


def _pool(rng, S, Hkv, spread=1.0):
    """A pool written earlier: (codes, scales) of k and v."""
    row = lambda: rng.standard_normal((S, Hkv, 64)) * np.exp(spread * rng.standard_normal((S, Hkv, 1)))  # noqa: E731
    return (*quantise(row()), *quantise(row()))


def _dev_pool(p):
    torch = _torch()
    kc, ks, vc, vs = (torch.from_numpy(x).cuda() for x in p)
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return kc.view(f8), vc.view(f8), ks.view(e8), vs.view(e8)


def _host_pool(d):
    torch = _torch()
    kc, vc, ks, vs = (x.view(torch.uint8).cpu().numpy() for x in d)
    return kc, ks, vc, vs


# ------------------------------------------------------------------ write

def _odd_rows(Hkv, dtype):
    """Rows at the edges: zeros, signs, ties, scales' limits, what is not finite."""
    f = np.zeros((24, Hkv, 64))
    f[1] = -0.0
    f[2, :, :] = np.linspace(-448, 448, 64)            # fills its scale exactly
    f[3] = 448.0
    f[4] = 450.0                                       # one power of two up
    f[5, :, ::2] = np.nan
    f[5, :, 1::2] = 3.0
    f[6] = np.inf
    f[7, :, 0], f[7, :, 1:] = -np.inf, 1.0
    f[8] = 1e-40
    f[9] = 2.0 ** -133
    f[10] = 3.3e38
    f[11, :, 0], f[11, :, 1:] = 3e38, 1e-30            # the small ones vanish
    for i in range(8):                                 # midpoints of neighbouring values
        mid = (VALUES[8 * i:8 * i + 64] + VALUES[8 * i + 1:8 * i + 65]) / 2
        f[12 + i] = np.where(np.isnan(mid), 0, mid)
        f[12 + i, :, 5] = 448.0
    f[20] = 2.0 ** -9 * np.arange(64)
    f[20, :, 0] = 448
    f[21] = -(2.0 ** -10)                              # its own scale lifts it
    f[22, :, 0], f[22, :, 1:] = 448.0, 2.0 ** -10      # a tie with zero
    f[23] = np.arange(64) - 31.5
    return _bits(f, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hkv", [(1, 8), (14, 8), (65, 3), (24, 1), (300, 16), (1001, 5), (4097, 2)])
def test_append_writes_the_nearest_values(n, Hkv, dtype):
    torch = _torch()
    rng = np.random.default_rng(n + Hkv)
    S = n + 9
    raw = rng.standard_normal((2, n, Hkv, 64)) * np.exp(4 * rng.standard_normal((2, n, Hkv, 1)))
    k, v = (_bits(x, dtype) for x in raw)
    if n >= 24:
        k[:24], v[n - 24:] = _odd_rows(Hkv, dtype), _odd_rows(Hkv, dtype)
    before = _pool(rng, S, Hkv)
    d = _dev_pool(before)
    slot = rng.permutation(S)[:n].astype(np.int32)
    slot[3::5] = rng.choice([-1, S, S + 7, -2 ** 31, 2 ** 31 - 1], slot[3::5].shape)  # padding
    # columns of one projection, with a gap
    x = torch.zeros(n, 2 * Hkv + 1, 64, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32,
                    device="cuda")
    x[:, :Hkv], x[:, Hkv + 1:] = akv.to_device(k, dtype), akv.to_device(v, dtype)
    akv.akv_append_kv_q8(akv.shape(max(1, Hkv), Hkv, 64, dtype), n, x[:, :Hkv], x[:, Hkv + 1:],
                         akv.i32_device(slot), *d)
    got = _host_pool(d)
    want = [x.copy() for x in before]
    real = (slot >= 0) & (slot < S)
    for y, a in ((k, 0), (v, 2)):
        want[a][slot[real]], want[a + 1][slot[real]] = quantise(_wide(y, dtype)[real])
    for a, name in enumerate(("k codes", "k scales", "v codes", "v scales")):
        g, w = got[a], want[a]
        if a % 2 == 0:  # NaN has two codes
            g, w = np.where(g % 128 == 127, 127, g), np.where(w % 128 == 127, 127, w)
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5])


def test_append_nothing_and_no_pool():
    torch = _torch()
    shp = akv.shape(8, 2)
    d = _dev_pool(_pool(np.random.default_rng(0), 4, 2))
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    akv.akv_append_kv_q8(shp, 0, rows[:0], rows[:0], akv.i32_device([]), *d)
    empty = [x[:0] for x in d]
    akv.akv_append_kv_q8(shp, 3, rows, rows, akv.i32_device([0, 1, 2]), *empty)
    torch.cuda.synchronize()


# ------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hkv", [(1, 8), (9, 3), (333, 8), (64, 16), (1000, 1), (77, 5)])
@pytest.mark.parametrize("turned", [False, True])
def test_read_back(n, Hkv, dtype, turned):
    """Values as they are held; keys rotated in fp32: angles good to 4e-7 and a
    few roundings of 2^-24, 2^-20 of the pair, and the output's rounding."""
    torch = _torch()
    rng = np.random.default_rng(n * 31 + Hkv)
    S, R = n + 5, n + 11
    p = _pool(rng, S, Hkv, 2.0)
    p[0][0, 0] = np.arange(64) * 2 % 127            # more of the codes
    p[2][0, 0], p[2][1, 0] = np.arange(64) + 63, np.arange(64) + 191
    p[2][(p[2] & 127) == 127] = 0
    d = _dev_pool(p)
    src, dst = rng.permutation(S)[:n].astype(np.int32), rng.permutation(R)[:n].astype(np.int32)
    src[0] = 0
    pos = rng.integers(-300000, 2000000, n).astype(np.int32)
    pos[: n // 2] = np.arange(n // 2)
    src[5::9], dst[7::9] = -1, R
    k_out = torch.full((R, Hkv, 64), 7.0, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    v_out = k_out.clone()
    akv.akv_read_kv_q8(akv.shape(Hkv, Hkv, 64, dtype), n, akv.i32_device(src),
                       akv.i32_device(pos) if turned else None, akv.i32_device(dst), *d, k_out, v_out)
    want_k, want_v = np.full((R, Hkv, 64), 7.0), np.full((R, Hkv, 64), 7.0)
    tol = np.zeros((R, Hkv, 64))
    ok = (src >= 0) & (dst < R)
    K, V = held(p[0], p[1])[src[ok]], held(p[2], p[3])[src[ok]]
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    Kt = turn(K, pos[ok]) if turned else K
    want_k[dst[ok]], want_v[dst[ok]] = Kt, V
    tol[dst[ok]] = u * np.abs(Kt) * (1 if turned else 0)
    if turned:
        tol[dst[ok]] += 2.0 ** -20 * (np.abs(K) + np.abs(np.roll(K, 32, -1)))
    got = k_out.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want_k) <= tol)
    assert np.array_equal(v_out.float().cpu().numpy().astype(np.float64), want_v)  # e4m3 fits in bf16


def test_read_every_code_and_scale():
    """All 256 codes under all scales that fp32 holds exactly, dst left out."""
    torch = _torch()
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(1, 4, 64), (255, 1, 1))
    scale = np.tile(np.arange(255, dtype=np.uint8)[:, None], (1, 4))
    d = _dev_pool((codes, scale, codes, scale))
    out = [torch.zeros(255, 4, 64, device="cuda") for _ in range(2)]
    akv.akv_read_kv_q8(akv.shape(4, 4, 64, "f32"), 255, akv.i32_device(np.arange(255)), None, None, *d, *out)
    with np.errstate(over="ignore"):  # 448 * 2^127 is no fp32 number
        want = held(codes, scale).astype(np.float32)
    for x in out:
        assert np.array_equal(x.cpu().numpy(), want, equal_nan=True)


# ----------------------------------------------------------------- decode

class Batch:
    def __init__(self, seed, n, Hq, Hkv, dtype, new=False, spread=1.0, scale=1.0, S=None, far=False):
        rng = np.random.default_rng(seed)
        self.n, self.Hq, self.Hkv, self.dtype, self.B = n, Hq, Hkv, dtype, len(n)
        self.ptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        nnz = int(self.ptr[-1])
        self.S = S or nnz + 7
        self.idx = rng.permutation(self.S)[:nnz].astype(np.int32)
        self.pos = rng.integers(0, 131072, nnz).astype(np.int32)
        for b in range(0, self.B, 2):  # in order, with gaps
            self.pos[self.ptr[b]:self.ptr[b + 1]] = np.arange(n[b]) + 97 * (np.arange(n[b]) // 31)
        if far:
            self.pos[::3] = rng.integers(-2 ** 30, 2 ** 30, len(self.pos[::3]))
        self.pool = [x.copy() for x in _pool(rng, self.S, Hkv, spread)]
        self.q = _bits(scale * rng.standard_normal((self.B, Hq, 64)), dtype)
        self.q_pos = rng.integers(0, 200000, self.B).astype(np.int32)
        self.new = new
        self.kn, self.vn = (_bits(rng.standard_normal((self.B, Hkv, 64)), dtype) for _ in range(2))
        self.slot = np.full(self.B, -1, np.int32)
        for b in range(self.B):
            if n[b]:
                self.slot[b] = self.idx[self.ptr[b + 1] - 1]
                if new:
                    self.q_pos[b] = self.pos[self.ptr[b + 1] - 1]
        self.shp, self.max_kv = akv.shape(Hq, Hkv, 64, dtype), max(n)

    def device(self):
        return dict(q=akv.to_device(self.q, self.dtype), pool=_dev_pool(self.pool),
                    kn=akv.to_device(self.kn, self.dtype), vn=akv.to_device(self.vn, self.dtype),
                    **{k: akv.i32_device(getattr(self, k)) for k in ("q_pos", "ptr", "idx", "pos", "slot")})

    def after(self):
        """The pool once the step's rows are in it."""
        p = [x.copy() for x in self.pool]
        if self.new:
            ok = (self.slot >= 0) & (self.slot < self.S) & (np.asarray(self.n) > 0)
            for x, a in ((self.kn, 0), (self.vn, 2)):
                p[a][self.slot[ok]], p[a + 1][self.slot[ok]] = quantise(_wide(x, self.dtype)[ok])
        return p

    def check(self, out, cut=None):
        p = self.after()
        K, V = held(p[0], p[1]), held(p[2], p[3])
        got = out.float().cpu().numpy().astype(np.float64)
        for b in range(self.B):
            r = slice(self.ptr[b], self.ptr[b] + (self.n[b] if cut is None else min(cut, self.n[b])))
            at = np.where((self.idx[r] >= 0) & (self.idx[r] < self.S), self.idx[r], 0)
            want, tol = decode(_wide(self.q, self.dtype)[b], self.q_pos[b], K[at], V[at], self.pos[r],
                               self.dtype)
            err = np.abs(got[b] - want)
            assert np.all(err <= tol), (b, float((err / np.maximum(tol, 1e-300)).max()))

    def workspace(self, max_kv=None):
        torch = _torch()
        return torch.full((akv.akv_decode_q8_workspace(self.shp, self.B, max_kv or self.max_kv),), 255,
                          dtype=torch.uint8, device="cuda")

    def run(self, d, max_kv=None, out=None, ws=None, stream=None):
        torch = _torch()
        out = torch.full_like(d["q"], 7.0) if out is None else out
        new = (d["kn"], d["vn"], d["slot"]) if self.new else (None, None, None)
        akv.akv_decode_attention_q8(self.shp, self.B, d["q"], d["q_pos"], *new, *d["pool"], d["ptr"], d["idx"],
                                    d["pos"], max_kv or self.max_kv, out,
                                    self.workspace(max_kv) if ws is None else ws, stream=stream)
        return out


LISTS = {"short": [1, 2, 15, 16, 17, 31, 33], "edges": [127, 0, 128, 129, 255, 257, 513],
         "one": [1], "mixed": [3000, 1, 700], "long": [20011, 9000]}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 4), (24, 3), (2, 2), (32, 16), (20, 1), (40, 2), (9, 1),
                                    (15, 5), (24, 24)])
@pytest.mark.parametrize("name", list(LISTS))
def test_decode(name, Hq, Hkv, dtype):
    torch = _torch()
    bt = Batch(len(name) + Hq, LISTS[name], Hq, Hkv, dtype, new=len(name) % 2 == 1)
    d = bt.device()
    out = bt.run(d)
    bt.check(out)
    assert all(np.array_equal(a, b) for a, b in zip(_host_pool(d["pool"]), bt.after()))
    assert torch.equal(out, bt.run(d))  # no order of atomics in it


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(16, 4), (24, 3), (20, 1)])
def test_decode_far_positions_and_slots_outside(Hq, Hkv, dtype):
    """Positions past 2^18 and below 0; list entries outside the pool read row 0;
    steps whose slot is outside it append nothing."""
    bt = Batch(3, [300, 41, 700], Hq, Hkv, dtype, new=True, far=True)
    bt.q_pos[1] = -123456789
    bt.idx[10], bt.idx[310], bt.idx[400] = -1, bt.S, 2 ** 31 - 1
    bt.slot[1] = bt.S + 3
    d = bt.device()
    bt.check(bt.run(d))
    assert all(np.array_equal(a, b) for a, b in zip(_host_pool(d["pool"]), bt.after()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ["peaky", "large queries", "large keys", "uneven values", "sink", "huge and tiny",
                                  "rising", "zeros"])
def test_decode_ranges(case, dtype):
    """Scores that jump, queries and keys past fp16's range, value rows of very
    different size (a weight of nearly 1 on a tiny value row beside many small
    weights on large ones)."""
    bt = Batch(17, [1500, 333], 16, 4, dtype, scale=16 if case == "peaky" else 1)
    wide = _wide(bt.q, dtype)
    kc, ks, vc, vs = bt.pool
    if case == "large queries":
        bt.q = _bits(wide * 2.0 ** 30, dtype)
        ks[:] = np.clip(ks.astype(int) - 30, 0, 254)
    elif case == "large keys":
        bt.q = _bits(wide * 2.0 ** -40, dtype)
        ks[:] = ks + 40
    elif case == "uneven values":
        vs[:] = np.clip(vs.astype(int) + np.random.default_rng(2).integers(-20, 21, vs.shape), 0, 254)
    elif case == "sink":
        first = bt.idx[bt.ptr[:-1]]
        bt.pos[:] = 0
        bt.q_pos[:] = 0
        q = np.zeros((2, 16, 64))
        q[..., 0] = 30.0
        bt.q = _bits(q, dtype)
        kc[...], ks[...] = quantise(np.zeros(kc.shape))
        k0 = np.zeros((2, 4, 64))
        k0[..., 0] = 5.0                       # a score 18.75 above the others'
        kc[first], ks[first] = quantise(k0)
        vs[first] -= 16
    elif case == "huge and tiny":
        vs[: len(vs) // 2], vs[len(vs) // 2:] = 200, 20
    elif case == "rising":
        bt.pos[:] = 0
        bt.q_pos[:] = 0
        q = np.zeros((2, 16, 64))
        q[..., 0] = 8.0
        bt.q = _bits(q, dtype)
        k0 = np.zeros((bt.idx.size, 4, 64))
        for b in range(2):
            j = np.arange(bt.n[b])
            k0[bt.ptr[b]:bt.ptr[b + 1], :, 0] = (j // 50 * 7.0)[:, None]
        kc[bt.idx], ks[bt.idx] = quantise(k0)
    elif case == "zeros":
        bt.q = _bits(0 * wide, dtype)
        vc[...], vs[...] = quantise(np.zeros(vc.shape))
    bt.check(bt.run(bt.device()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_bounds_and_what_is_not_listed(dtype):
    """Lists longer than max_kv are cut to it; one shorter leaves the answer as it
    is; rows of the pool that no list names may hold anything; a batch of none."""
    torch = _torch()
    bt = Batch(23, [700, 40, 0, 65], 24, 3, dtype)
    idle = np.setdiff1d(np.arange(bt.S), bt.idx)
    bt.pool[0][idle], bt.pool[2][idle], bt.pool[1][idle], bt.pool[3][idle] = 127, 255, 255, 255
    if 0 in bt.idx:  # row 0 stands in for slots outside the pool and past the lists
        pass
    d = bt.device()
    full = bt.run(d)
    bt.check(full)
    assert not full[2].any()
    bt.check(bt.run(d, max_kv=5000))
    bt.check(bt.run(d, max_kv=100), cut=100)
    empty = torch.empty(0, 24, 64, dtype=d["q"].dtype, device="cuda")
    none = akv.i32_device([])
    akv.akv_decode_attention_q8(bt.shp, 0, empty, none, None, None, None, *d["pool"], akv.i32_device([0]), none,
                                none, 0, empty, None)
    # requests, but no list has an entry and no pool a row
    out = torch.full((2, 24, 64), 7.0, dtype=d["q"].dtype, device="cuda")
    ws = torch.empty(akv.akv_decode_q8_workspace(bt.shp, 2, 64), dtype=torch.uint8, device="cuda")
    akv.akv_decode_attention_q8(bt.shp, 2, out.clone(), akv.i32_device([0, 1]), None, None, None,
                                *[x[:0] for x in d["pool"]], akv.i32_device([0, 0, 0]), none, none, 64, out, ws)
    assert not out.any()


def test_decode_nan_reaches_only_its_own():
    """A NaN that a list names reaches that request's head group and no other."""
    bt = Batch(29, [300, 300], 16, 4, "bf16")
    bt.pool[2][bt.idx[20], 1, 5] = 127
    d = bt.device()
    got = bt.run(d).float().cpu().numpy()
    hit = np.zeros((2, 16, 64), bool)
    hit[0, 4:8, 5] = True
    assert np.array_equal(np.isnan(got), hit)


def test_decode_offsets_past_32_bits():
    """4.3 million slots of 8 heads: codes past 2^31."""
    torch = _torch()
    S, Hq, Hkv = 4_300_000, 16, 8
    bt = Batch(31, [40, 200], Hq, Hkv, "bf16", S=300)
    big = S - 300
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    pool = [torch.zeros(S, Hkv, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.zeros(S, Hkv, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, y in zip((*pool, *scale), (bt.pool[0], bt.pool[2], bt.pool[1], bt.pool[3])):
        x[big:] = torch.from_numpy(y).cuda()
    d = bt.device()
    d["idx"] = d["idx"] + big
    d["pool"] = (pool[0].view(f8), pool[1].view(f8), scale[0].view(e8), scale[1].view(e8))
    bt.check(bt.run(d))
    # read back and written there too
    k, v = (torch.zeros(300, Hkv, 64, device="cuda") for _ in range(2))
    shp = akv.shape(Hkv, Hkv, 64, "f32")
    at = akv.i32_device(np.arange(big, S))
    akv.akv_read_kv_q8(shp, 300, at, None, None, *d["pool"], k, v)
    assert np.array_equal(k.cpu().numpy(), held(bt.pool[0], bt.pool[1]).astype(np.float32))
    akv.akv_append_kv_q8(shp, 300, 2 * k, 2 * v, at, *d["pool"])
    akv.akv_read_kv_q8(shp, 300, at, None, None, *d["pool"], k, v)
    assert np.array_equal(v.cpu().numpy(), 2 * held(bt.pool[2], bt.pool[3]).astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_captured_and_on_two_streams(dtype):
    """A captured step replays for other lists within its bounds; two streams, a
    workspace each, do not disturb one another."""
    torch = _torch()
    a = Batch(37, [900, 50, 300], 24, 3, dtype, new=True)
    b = Batch(38, [10, 899, 2], 24, 3, dtype, new=True, S=a.S)
    d, e = a.device(), b.device()
    a.run(d, max_kv=900)
    ws, out = a.workspace(900), torch.zeros_like(d["q"])
    # room for either batch's lists
    n = max(d["idx"].numel(), e["idx"].numel())
    for x in (d, e):
        for k in ("idx", "pos"):
            x[k] = torch.cat([x[k], x[k].new_zeros(n - x[k].numel())])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(d, max_kv=900, out=out, ws=ws)
    g.replay()
    a.check(out)
    flat = lambda x: [y for v in x.values() for y in (v if isinstance(v, tuple) else (v,))]  # noqa: E731
    for x, y in zip(flat(d), flat(e)):
        x.view(torch.uint8).copy_(y.view(torch.uint8))
    g.replay()
    b.check(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    bts = [Batch(40 + i, [5000 + i, 700], 24, 3, dtype) for i in range(2)]
    ds = [x.device() for x in bts]
    wss, outs = [x.workspace() for x in bts], [torch.zeros_like(x["q"]) for x in ds]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            bts[i].run(ds[i], out=outs[i], ws=wss[i], stream=s)
    torch.cuda.synchronize()
    for bt, o in zip(bts, outs):
        bt.check(o)


def test_binding_refuses():
    torch = _torch()
    bt = Batch(43, [30], 16, 4, "bf16")
    d = bt.device()
    for k, bad in (("q", d["q"].float()), ("pos", d["pos"].long()), ("ptr", d["ptr"][:1]), ("idx", d["idx"].cpu())):
        with pytest.raises(ValueError):
            bt.run({**d, k: bad})
    with pytest.raises(ValueError):
        bt.run({**d, "pool": (d["pool"][0].view(torch.uint8), *d["pool"][1:])})
    with pytest.raises(ValueError):
        bt.run({**d, "pool": (*d["pool"][:2], d["pool"][2][:-1], d["pool"][3])})
    with pytest.raises(akv.AkvError) as e:
        bt.run(d, ws=bt.workspace()[:-256] if bt.workspace().numel() > 256 else bt.workspace()[:1])
    assert "WORKSPACE" in str(e.value)


@pytest.mark.parametrize("Hq,Hkv", [(12, 12), (40, 20), (12, 6), (14, 7), (30, 10), (22, 11), (100, 4)])
def test_decode_head_counts_that_split_scale_words(Hq, Hkv):
    """KV heads whose scales do not fill whole words, that take several CTAs, the
    last of them with fewer heads; a pool whose last rows' words end with it."""
    bt = Batch(50 + Hkv, [700, 33, 1, 129], Hq, Hkv, "bf16", new=True, S=870)
    bt.idx[5], bt.idx[700] = bt.S - 1, bt.S - 1  # the pool's last row, twice
    bt.slot[:] = [bt.idx[p - 1] for p in bt.ptr[1:]]
    if bt.S - 1 in bt.slot:
        bt.new = False
    d = bt.device()
    bt.check(bt.run(d))
    assert all(np.array_equal(a, b) for a, b in zip(_host_pool(d["pool"]), bt.after()))


def test_decode_many_requests():
    """700 short lists, every fifth empty: ranges that hold several requests."""
    rng = np.random.default_rng(5)
    n = [0 if b % 5 == 2 else int(rng.integers(1, 90)) for b in range(700)]
    for Hq, Hkv in ((16, 8), (4, 1)):
        bt = Batch(60, n, Hq, Hkv, "bf16", new=True)
        d = bt.device()
        bt.check(bt.run(d))
        assert all(np.array_equal(a, b) for a, b in zip(_host_pool(d["pool"]), bt.after()))
