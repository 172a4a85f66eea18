"""The 8-bit decode's cut of the lists and its precision, by comparisons that a lost or
repeated tile or a lost part of the query passes (test_kv8_sharp_host.py plants them)."""
import numpy as np
import pytest

import kv_cache_drop_gb300 as akv
from _kv8 import held, quantise
from _kv8_sharp import SPREAD, decode_norm, flat_scores, modest_pool, unit_values
from test_gpu_kv8 import LISTS, Batch, _bits, _wide

pytestmark = pytest.mark.gpu

MANY = [0 if b % 5 == 2 else 1 + 37 * b % 113 for b in range(400)]
SHARP = {**LISTS, "many": MANY}


def _check_norms(bt, out, **how):
    p = bt.after()
    K, V, q = held(p[0], p[1]), held(p[2], p[3]), _wide(bt.q, bt.dtype)
    got = out.float().cpu().numpy().astype(np.float64)
    for b in range(bt.B):
        r = slice(bt.ptr[b], bt.ptr[b + 1])
        want, bound = decode_norm(q[b], bt.q_pos[b], K[bt.idx[r]], V[bt.idx[r]], bt.pos[r], **how)
        off = np.linalg.norm(got[b] - want, axis=1)
        assert np.all(off <= bound), (b, float((off / np.maximum(bound, 1e-300)).max()))


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 4), (24, 3), (2, 2), (20, 1), (40, 2), (40, 20)])
@pytest.mark.parametrize("name", list(SHARP))
def test_norm_of_each_head(name, Hq, Hkv):
    bt = Batch(101 + Hq, SHARP[name], Hq, Hkv, "bf16", new=len(name) % 2 == 0, scale=SPREAD)
    bt.pool = modest_pool(np.random.default_rng(Hkv), bt.S, Hkv)
    _check_norms(bt, bt.run(bt.device()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 4), (24, 3), (2, 2), (20, 1), (9, 1), (12, 12), (40, 20), (100, 4)])
@pytest.mark.parametrize("name", list(SHARP))
def test_every_entry_counts_once(name, Hq, Hkv, dtype):
    """A query of zeros: all weights are equal and exact, and an output component is the
    count of its run of entries over the list's length, rounded: to 2^-8 of it in bf16,
    and twice to 2^-24 for the quotient in fp32."""
    bt = Batch(7, SHARP[name], Hq, Hkv, dtype, new=True)
    bt.q = _bits(np.zeros((bt.B, Hq, 64)), dtype)
    V = np.concatenate([unit_values(n, Hkv) for n in bt.n])
    bt.pool[2][...], bt.pool[3][...] = 0, 0
    bt.pool[2][bt.idx], bt.pool[3][bt.idx] = quantise(V)
    last = np.maximum(bt.ptr[1:] - 1, 0)
    bt.vn = _bits(V[last], dtype)  # the step's row is its list's last entry
    got = bt.run(bt.device()).float().cpu().numpy().astype(np.float64)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    for b, n in enumerate(bt.n):
        want = V[bt.ptr[b]:bt.ptr[b + 1]].sum(0) / max(n, 1)
        want = np.repeat(want, Hq // Hkv, 0)
        assert np.all(np.abs(got[b] - want) <= 1.001 * u * want), (b, n, float(np.abs(got[b] - want).max() * n))


@pytest.mark.parametrize("Hkv", [1, 2, 8])
def test_both_parts_of_the_query(Hkv):
    """Scores of some hundred terms each, whose sums are within 1.5 of one another."""
    n = 1500
    q, q_pos, kc, ks = flat_scores(11 + Hkv, Hkv, n)
    bt = Batch(12, [n], Hkv, Hkv, "bf16")
    bt.pool = modest_pool(np.random.default_rng(13), bt.S, Hkv)
    bt.pool[0][bt.idx], bt.pool[1][bt.idx] = kc, ks
    bt.q, bt.q_pos, bt.pos = _bits(q[None], "bf16"), np.array([q_pos], np.int32), np.zeros(n, np.int32)
    assert np.array_equal(_wide(bt.q, "bf16")[0], q)
    _check_norms(bt, bt.run(bt.device()), rotated=False, terms=2.0 ** -22)


def test_ranges_of_a_replayed_call():
    """A captured call replayed for lists of other lengths cuts them anew."""
    import torch
    Hq, Hkv = 16, 8
    lists = [[9000, 1, 40], [1, 9000, 40], [3000, 3041, 3000], [0, 9041, 0], [5, 0, 33]]
    bts = []
    for n in lists:
        bt = Batch(31, n, Hq, Hkv, "bf16", S=9100)
        bt.q = _bits(np.zeros((3, Hq, 64)), "bf16")
        bt.V = np.concatenate([unit_values(x, Hkv) for x in n])
        bt.pool[2][...], bt.pool[3][...] = 0, 0
        bt.pool[2][bt.idx], bt.pool[3][bt.idx] = quantise(bt.V)
        bts.append(bt)
    ds = [bt.device() for bt in bts]
    room = dict(ds[0])
    ws, out = bts[0].workspace(9041), torch.zeros_like(room["q"])
    bts[0].run(room, max_kv=9041, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bts[0].run(room, max_kv=9041, out=out, ws=ws)
    for bt, d in zip(bts, ds):
        for k in ("ptr", "idx", "pos"):
            room[k][:d[k].numel()].copy_(d[k])
        for x, y in zip(room["pool"], d["pool"]):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        g.replay()
        got = out.float().cpu().numpy().astype(np.float64)
        for b, n in enumerate(bt.n):
            want = np.repeat(bt.V[bt.ptr[b]:bt.ptr[b + 1]].sum(0) / max(n, 1), Hq // Hkv, 0)
            assert np.all(np.abs(got[b] - want) <= 1.001 * 2.0 ** -8 * want), (bt.n, b)
    assert akv.akv_decode_q8_workspace(bts[0].shp, 3, 9041) == ws.numel()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lists_inside_longer_arrays(dtype):
    """kv_indptr need not begin at 0 nor the arrays end with the last list: entries
    before and behind name rows of NaN."""
    import torch
    bt = Batch(41, [900, 0, 33, 2100], 24, 3, dtype, new=True)
    bt.pool = modest_pool(np.random.default_rng(2), bt.S, 3)
    spare = np.setdiff1d(np.arange(bt.S), bt.idx)[:1]
    bt.pool[0][spare], bt.pool[2][spare] = 127, 127
    d = bt.device()
    before = bt.run(d)
    bt.check(before)
    e = bt.device()
    pad = lambda x, lo, hi: torch.cat([x.new_full((lo,), int(spare[0])), x, x.new_full((hi,), int(spare[0]))])  # noqa: E731
    e["idx"], e["pos"], e["ptr"] = pad(e["idx"], 1237, 70), pad(e["pos"], 1237, 70), e["ptr"] + 1237
    after = bt.run(e)
    bt.check(after)
    assert torch.equal(before, after)
