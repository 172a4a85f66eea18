"""The 8-bit decode's workspace serves every smaller call (no GPU)."""
import random

import pytest

from test_chunk_host import akv  # noqa: F401


def _need(akv, shp, B, max_kv):  # noqa: F811
    n = akv.akv_decode_q8_workspace(shp, B, max_kv)
    assert n > 0
    return n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (16, 4), (2, 2), (24, 3), (100, 1), (40, 20)])
def test_neighbouring_bounds(akv, Hq, Hkv, dtype):  # noqa: F811
    """Around every multiple of 128 entries, where the cut of the lists changes (a
    batch of 14 over 5,376 entries took finer splits than one over 5,632), and around
    every batch size."""
    shp = akv.shape(Hq, Hkv, 64, dtype)
    last = 0
    for n in sorted({128 * i + d for i in range(0, 400) for d in (0, 1)} |
                    {2 ** i + d for i in range(15, 30) for d in (-1, 0, 1)}):
        now = _need(akv, shp, 14, n)
        assert now >= last, n
        last = now
    for n in (1, 700, 5376, 90000, 1 << 30):
        sizes = [_need(akv, shp, B, n) for B in [*range(1, 300), 1000, 65535]]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_any_smaller_call(akv, dtype):  # noqa: F811
    rng = random.Random(7)
    for _ in range(3000):
        Hkv = rng.choice([1, 2, 3, 8, 20, 64])
        shp = akv.shape(Hkv * rng.choice([1, 8, 17]), Hkv, 64, dtype)
        B, n = int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 30))
        b, m = rng.randint(1, B), rng.randint(0, n)
        assert _need(akv, shp, b, m) <= _need(akv, shp, B, n), (Hkv, B, n, b, m)
