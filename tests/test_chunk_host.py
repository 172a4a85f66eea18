"""Host-side checks of the calls over a chunk of new tokens (no GPU): what is
refused before anything is enqueued, and the workspace sizes.  Addresses are
made up; a refused call never reads them."""
import ctypes
import math
import os

import pytest

OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 3, 4
P = 1 << 20  # a 16- and 256-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def akv():
    import kv_cache_drop_gb300 as m
    from kv_cache_drop_gb300 import _build
    if not os.path.exists(m.LIB_PATH):
        _build.build()
    m.lib()
    return m


def _call(akv, fn, defaults, **change):
    args = dict(defaults)
    for k in change:
        assert k in args, k
    args.update(change)
    a = [ctypes.byref(v) if isinstance(v, akv.Shape) else v for v in args.values()]
    return getattr(akv.lib(), fn)(*a)


def _append(akv, **change):
    return _call(akv, "akv_qk_norm_append", dict(
        shape=akv.shape(8, 2), n=3, q=P, qs=512, k=P, ks=128, v=P, vs=128, qw=None, kw=None,
        eps=1e-6, flags=15, pos=P, slot=P, S=10, q_out=2 * P, kp=P, vp=P, stream=None), **change)


def _chunk(akv, **change):
    return _call(akv, "akv_chunk_attention", dict(
        shape=akv.shape(8, 2), B=2, q_indptr=P, n_rows=4, max_q=3, q=P, kp=P, vp=P, S=100,
        kv_indptr=P, kv_indices=P, max_kv=50, out=P, lse=P, ws=P, ws_bytes=1 << 30, stream=None),
        **change)


def _mass(akv, **change):
    return _call(akv, "akv_attention_mass", dict(
        shape=akv.shape(8, 2), B=2, q_indptr=P, n_rows=4, max_q=3, q=P, kp=P, S=100, kv_indptr=P,
        kv_indices=P, max_kv=50, lse=P, decay=1.0, mass_in=P, mass_out=P, stride=50, ws=P,
        ws_bytes=1 << 30, stream=None), **change)


def _evict(akv, **change):
    return _call(akv, "akv_evict_by_mass", dict(
        B=2, kv_indptr=P, kv_indices=P, kv_pos=P, max_kv=50, mass=P, stride=50, keep=P, n_first=1,
        n_recent=1, out_indptr=P, out_indices=P, out_pos=P, out_mass=2 * P, out_stride=50,
        out_cap=100, dropped_indptr=P, dropped=P, dropped_cap=100, stream=None), **change)


def test_append_refusals(akv):
    for change in (dict(n=-1), dict(S=-1), dict(flags=16), dict(flags=-1), dict(eps=-1.0),
                   dict(eps=math.nan), dict(eps=math.inf), dict(q=None), dict(k=None),
                   dict(v=None), dict(slot=None), dict(pos=None), dict(q_out=None), dict(kp=None),
                   dict(vp=None), dict(qs=511), dict(qs=504), dict(ks=120), dict(vs=127),
                   dict(qs=516), dict(ks=132), dict(q=P + 8), dict(k=P + 2), dict(v=P + 4),
                   dict(q_out=P + 8), dict(kp=P + 8), dict(vp=P + 8),
                   dict(q_out=P, qs=1024), dict(shape=akv.shape(7, 2))):
        assert _append(akv, **change) == INVALID, change
        assert akv.lib().akv_last_error()
    assert _append(akv, shape=akv.shape(8, 2, 128)) == UNSUPPORTED
    assert _append(akv, n=0, q=None, k=None) == OK
    # fp32 rows: strides in multiples of 4 elements
    f32 = akv.shape(8, 2, 64, "f32")
    assert _append(akv, shape=f32, qs=514) == INVALID


def test_chunk_refusals(akv):
    for change in (dict(B=-1), dict(n_rows=-1), dict(max_q=-1), dict(max_kv=-1), dict(S=-1),
                   dict(S=0), dict(q_indptr=None), dict(q=None), dict(kp=None), dict(vp=None),
                   dict(kv_indptr=None), dict(kv_indices=None), dict(out=None), dict(q=P + 8),
                   dict(kp=P + 2), dict(vp=P + 2), dict(out=P + 8), dict(shape=akv.shape(7, 2))):
        assert _chunk(akv, **change) == INVALID, change
        assert akv.lib().akv_last_error()
    for change in (dict(B=65536), dict(max_kv=(1 << 30) + 1), dict(shape=akv.shape(8, 2, 128)),
                   dict(shape=akv.shape(65536, 1)),
                   dict(max_q=2**31 - 1, n_rows=2**31 - 1, shape=akv.shape(4096, 1))):
        assert _chunk(akv, **change) == UNSUPPORTED, change
    for change in (dict(B=0), dict(n_rows=0, q=None), dict(max_q=0)):
        assert _chunk(akv, **change) == OK, change
    need = akv.akv_chunk_workspace(akv.shape(8, 2), 2, 4, 3, 50000)
    assert need > 0
    for change in (dict(ws=None), dict(ws=P + 128), dict(ws_bytes=need - 1)):
        assert _chunk(akv, max_kv=50000, **change) == WORKSPACE, change


def test_mass_refusals(akv):
    for change in (dict(B=-1), dict(n_rows=-1), dict(max_q=-1), dict(max_kv=-1), dict(S=-1),
                   dict(S=0), dict(q_indptr=None), dict(q=None), dict(lse=None), dict(kp=None),
                   dict(kv_indptr=None), dict(kv_indices=None), dict(mass_out=None),
                   dict(stride=49), dict(decay=math.nan), dict(decay=math.inf), dict(q=P + 8),
                   dict(kp=P + 8), dict(shape=akv.shape(7, 2))):
        assert _mass(akv, **change) == INVALID, change
        assert akv.lib().akv_last_error()
    for change in (dict(B=65536), dict(max_kv=(1 << 30) + 1, stride=1 << 31),
                   dict(shape=akv.shape(8, 2, 128))):
        assert _mass(akv, **change) == UNSUPPORTED, change
    for change in (dict(B=0), dict(max_kv=0)):
        assert _mass(akv, **change) == OK, change
    need = akv.akv_attention_mass_workspace(akv.shape(64, 8), 1, 4096, 4096, 4096)
    if need:
        big = dict(shape=akv.shape(64, 8), B=1, n_rows=4096, max_q=4096, max_kv=4096, stride=4096)
        for change in (dict(ws=None), dict(ws=P + 128), dict(ws_bytes=need - 1)):
            assert _mass(akv, **big, **change) == WORKSPACE, change


def test_evict_refusals(akv):
    for change in (dict(B=-1), dict(max_kv=-1), dict(n_first=-1), dict(n_recent=-1),
                   dict(stride=49), dict(out_stride=-1), dict(out_cap=-1), dict(dropped_cap=-1),
                   dict(kv_indptr=None), dict(keep=None), dict(out_indptr=None),
                   dict(dropped_indptr=None), dict(kv_indices=None), dict(mass=None),
                   dict(out_indices=None), dict(out_mass=None), dict(dropped=None),
                   dict(kv_pos=None), dict(out_pos=None), dict(out_mass=P)):
        assert _evict(akv, **change) == INVALID, change
        assert akv.lib().akv_last_error()
    for change in (dict(B=65536), dict(max_kv=(1 << 30) + 1, stride=1 << 31)):
        assert _evict(akv, **change) == UNSUPPORTED, change
    assert _evict(akv, B=0) == OK


def test_workspace_queries_refuse_nonsense(akv):
    L = akv.lib()
    for f in (L.akv_chunk_workspace, L.akv_attention_mass_workspace):
        assert f(None, 1, 1, 1, 1) == 0
        for bad in ((0, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, -1)):
            assert f(ctypes.byref(akv.shape(8, 2)), *bad) == 0
