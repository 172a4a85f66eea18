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
