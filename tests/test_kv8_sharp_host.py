"""The sharper tests' bounds, on the CPU: faults planted in the definition pass them."""
import numpy as np
import pytest

from _kv8 import held, turn
from _kv8_sharp import SPREAD, decode_norm, flat_scores, modest_pool, unit_values

LISTS = {"short": [1, 2, 15, 16, 17, 31, 33], "edges": [127, 128, 129, 255, 257, 513], "mixed": [3000, 1, 700],
         "long": [20011, 9000]}


@pytest.mark.parametrize("name", list(LISTS))
def test_a_fault_passes_the_bound(name):
    """An output of zeros, a tile of 32 left out or counted twice (the first, one in the
    middle, the last): each is off by more than twice the bound, at every length.  The
    scores' spread is small, so that no entry hides the others."""
    rng = np.random.default_rng(len(name))
    for n in LISTS[name]:
        kc, ks, vc, vs = modest_pool(rng, n, 2)
        K, V = held(kc, ks), held(vc, vs)
        q, pos = SPREAD * rng.standard_normal((8, 64)), rng.integers(0, 131072, n)
        want, bound = decode_norm(q, 777, K, V, pos)
        assert np.all(np.linalg.norm(want, axis=1) > 2 * bound)
        tiles = (n + 31) // 32
        for t in {0, tiles // 2, tiles - 1}:
            for times in (0, 2):
                if tiles == 1:
                    continue
                kept = np.ones(n)
                kept[32 * t:32 * t + 32] = times
                got, _ = decode_norm(q, 777, K, V, pos, kept)
                off = np.linalg.norm(got - want, axis=1) / bound
                assert np.max(off) > 2, (n, t, times, off)


def test_the_query_s_second_part():
    """The query rounded to 11 bits is off by more than twice the bound."""
    q, q_pos, kc, ks = flat_scores(3, 2, 1500)
    K = held(kc, ks)
    V = np.random.default_rng(4).standard_normal((1500, 2, 64))
    pos = np.zeros(1500, np.int64)
    want, bound = decode_norm(q, q_pos, K, V, pos, rotated=False, terms=2.0 ** -22)
    qr = turn(q[None], [q_pos])[0]
    got, _ = decode_norm(qr.astype(np.float16).astype(np.float64), 0, K, V, pos, rotated=False)
    assert np.all(np.linalg.norm(got - want, axis=1) > 2 * bound)


@pytest.mark.parametrize("n,Hkv", [(1, 1), (129, 3), (3000, 2), (20011, 8), (20011, 1)])
def test_units(n, Hkv):
    """Each entry has one component, and an entry more or less of a run of up to 100
    passes twice the rounding of 2^-8."""
    v = unit_values(n, Hkv)
    counts = v.sum(0)
    assert counts.sum() == n and np.all(v.sum((1, 2)) == 1)
    run = counts.max()
    if run <= 100:
        assert 1 / run > 2 * 2.0 ** -8
    assert 32 / run > 2 * 2.0 ** -8  # a tile
