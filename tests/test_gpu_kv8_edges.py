"""The 8-bit cache where it can go wrong: a workspace sized for larger calls, value
rows of very different size, positions near the ends of int32, lists left out."""
import fractions
import math

import numpy as np
import pytest

import kv_cache_drop_gb300 as akv
from _kv8 import held, quantise
from test_gpu_kv8 import Batch, _bits, _dev_pool, _wide

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


# -------------------------------------------------------------- workspace

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_workspace_serves_smaller_calls(dtype):
    """14 requests over up to 5,376 entries in the workspace of 5,632, and 13 in
    that of 14; nothing behind it is written."""
    torch = _torch()
    bt = Batch(71, [5376 - 300 * b for b in range(14)], 8, 8, dtype)
    d = bt.device()
    need = akv.akv_decode_q8_workspace(bt.shp, 14, 5632)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = bt.run(d, max_kv=5376, ws=room[:need])
    bt.check(out)
    few = Batch(72, bt.n[:13], 8, 8, dtype)
    e = few.device()
    few.check(few.run(e, max_kv=5376, ws=room[:need]))
    few.check(few.run(e, max_kv=5632, ws=room[:need]))
    assert bool((room[need:] == 77).all())


# ----------------------------------------------------------------- values

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (64, 8), (80, 8), (9, 1)])
@pytest.mark.parametrize("power", [20, 28, 60, 115])
def test_a_large_value_row_without_weight(power, Hq, Hkv, dtype):
    """Entries in threes of tiles: value rows of zeros, which have the smallest scale;
    then more of these and among them rows of up to 448 * 2^power whose weight is
    exp(-320); then ordinary rows, whose part is all of the output.

    Every score is exact: positions are 0, the query and the keys have one component.
    The output is sum w v / sum w over the rows of weight 1 and exp(-1), whose sums
    are good to 2^-18 in fp32, with weights rounded to fp16 (2^-11 each) and, in
    bf16, the output to 2^-8 of itself.  What the large rows put in is below
    448 * 2^115 exp(-320) = 2^-338."""
    n = 3 * 3 * 256
    bt = Batch(73, [n, n // 3 + 5], Hq, Hkv, dtype)
    bt.pos[:], bt.q_pos[:] = 0, 0
    q = np.zeros((2, Hq, 64))
    q[..., 0] = 64.0
    bt.q = _bits(q, dtype)
    kc, ks, vc, vs = bt.pool
    rng = np.random.default_rng(power)
    for b in range(2):
        rows = bt.idx[bt.ptr[b]:bt.ptr[b + 1]]
        j = np.arange(len(rows))
        kind = j // 256 % 3  # zeros, large, ordinary
        kind[(kind == 1) & (j % 7 != 3)] = 0
        k = np.zeros((len(rows), Hkv, 64))
        k[..., 0] = np.where(kind == 1, -40.0, np.where(kind == 2, -0.125, 0.0))[:, None]
        v = rng.standard_normal((len(rows), Hkv, 64)) + 2
        v[kind == 0] = 0
        v[kind == 1] *= 2.0 ** power
        kc[rows], ks[rows] = quantise(k)
        vc[rows], vs[rows] = quantise(v)
    got = bt.run(bt.device()).float().cpu().numpy().astype(np.float64)
    V = held(vc, vs)
    for b in range(2):
        rows = bt.idx[bt.ptr[b]:bt.ptr[b + 1]]
        s = 8 * held(kc, ks)[rows][..., 0]                      # [n, Hkv]
        w = np.exp(s)
        want = np.einsum("jg,jgd->gd", w, V[rows]) / w.sum(0)[:, None]
        size = np.einsum("jg,jgd->gd", w, np.abs(V[rows])) / w.sum(0)[:, None]
        want, size = np.repeat(want, Hq // Hkv, 0), np.repeat(size, Hq // Hkv, 0)
        tol = (2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -18) * size if dtype == "bf16"
               else 2.0 ** -24 * np.abs(want) + 2.0 ** -18 * size)
        assert np.all(np.abs(got[b] - want) <= tol), float(np.abs((got[b] - want) / tol).max())


# -------------------------------------------------------------- positions

# 2 pi to 70 digits
TWO_PI = fractions.Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632")


def _turned(theta, pos):
    """theta * pos modulo 2 pi, in -pi .. pi."""
    x = fractions.Fraction(theta) * pos
    x -= round(x / TWO_PI) * TWO_PI
    return float(x)


@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_angles_of_far_positions(base):
    """Positions near both ends of int32 at which one frequency's angle is next to a
    whole turn, so that its sine shows the angle's own error.

    The frequency is a double.  Its turn is a product in integers, off by at most one
    of 2^-32 turns for the floor and, for the frequency's rounding to 2^-64 turns,
    2^31 * 2^-65 = a quarter of 2^-32 more: by less than 1.3 * 2 pi * 2^-32 < 1.91e-9.
    The turn's conversion to fp32 and the sine and cosine are good to four roundings
    of 2^-24 relative to them."""
    torch = _torch()
    n = 32
    thetas = [math.pow(float(np.float32(base)), -2.0 * f / 64) for f in range(n)]
    pos, rng = [], np.random.default_rng(5)
    for f in range(n):
        best = []
        for sign in (-1, 1):
            tries = [sign * (2 ** 31 - 2 - int(x)) for x in rng.integers(0, 2 ** 20, 4000)]
            best.append(min(tries, key=lambda p: abs(math.remainder(thetas[f] * p, 2 * math.pi))))
        pos += best
    pos = np.array(pos, np.int64)
    codes = np.zeros((2 * n, 1, 64), np.uint8)
    codes[..., :32] = 0x38                                      # 1.0
    scale = np.full((2 * n, 1), 127, np.uint8)
    d = _dev_pool((codes, scale, codes, scale))
    out = [torch.zeros(2 * n, 1, 64, device="cuda") for _ in range(2)]
    akv.akv_read_kv_q8(akv.shape(1, 1, 64, "f32", base), 2 * n, akv.i32_device(np.arange(2 * n)),
                       akv.i32_device(pos.astype(np.int32)), None, *d, *out)
    got = out[0].cpu().numpy().astype(np.float64)[:, 0]
    for i, p in enumerate(pos):
        f = i // 2
        a = _turned(thetas[f], int(p))
        assert abs(got[i, f + 32] - math.sin(a)) <= 1.91e-9 + 2.0 ** -22 * abs(math.sin(a)), (f, int(p), a)
        assert abs(got[i, f] - math.cos(a)) <= 1.91e-9 + 2.0 ** -22, (f, int(p), a)


# ------------------------------------------------------------ lists left out

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lists_and_pool_left_out(dtype):
    """Where max_kv is 0 the lists may be None: every request gets zeros."""
    torch = _torch()
    bt = Batch(75, [3, 4], 16, 4, dtype)
    d = bt.device()
    out = torch.full_like(d["q"], 7.0)
    ws = torch.empty(akv.akv_decode_q8_workspace(bt.shp, 2, 0), dtype=torch.uint8, device="cuda")
    akv.akv_decode_attention_q8(bt.shp, 2, d["q"], d["q_pos"], None, None, None, *d["pool"], d["ptr"], None, None, 0,
                                out, ws)
    assert not out.any()
    with pytest.raises(akv.AkvError):
        akv.akv_decode_attention_q8(bt.shp, 2, d["q"], d["q_pos"], None, None, None, *d["pool"], d["ptr"], None,
                                    None, 5, out, ws)
    with pytest.raises(ValueError):
        akv.akv_decode_attention_q8(bt.shp, 2, d["q"], d["q_pos"], None, None, None, *d["pool"], d["ptr"], d["idx"],
                                    d["pos"][:-1], 4, out, ws)
    assert np.array_equal(_wide(bt.q, dtype), d["q"].float().cpu().numpy())
    # the chunk calls' lists as well
    ptr = akv.i32_device([0, 1, 2])
    lse = torch.zeros(2, 16, device="cuda")
    pool = torch.zeros(3, 4, 64, dtype=d["q"].dtype, device="cuda")
    ws = torch.empty(akv.akv_chunk_workspace(bt.shp, 2, 2, 1, 0), dtype=torch.uint8, device="cuda")
    out.fill_(7.0)
    akv.akv_chunk_attention(bt.shp, 2, ptr, d["q"], pool, pool, d["ptr"], None, 1, 0, out, lse, ws)
    assert not out.any() and bool(torch.isneginf(lse).all())
