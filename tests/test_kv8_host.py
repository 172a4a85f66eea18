"""Host-side checks of the 8-bit cache's and the shared prefix's calls (no GPU):
what is refused before anything is enqueued, and the workspace sizes.  Addresses
are made up; a refused call never reads them."""
import ctypes

import numpy as np
import pytest

from _kv8 import VALUES, held, quantise
from test_chunk_host import INVALID, OK, P, UNSUPPORTED, WORKSPACE, _call, akv  # noqa: F401


def _append(akv, **change):  # noqa: F811
    return _call(akv, "akv_append_kv_q8", dict(
        shape=akv.shape(8, 2), n=3, k=P, ks=128, v=P, vs=128, slot=P, S=10, kp=P, vp=P, k_scale=P, v_scale=P,
        stream=None), **change)


def _read(akv, **change):  # noqa: F811
    return _call(akv, "akv_read_kv_q8", dict(
        shape=akv.shape(8, 2), n=3, src=P, pos=P, dst=P, kp=P, vp=P, k_scale=P, v_scale=P, S=10, k_out=P, v_out=P,
        R=5, stream=None), **change)


def _decode(akv, **change):  # noqa: F811
    return _call(akv, "akv_decode_attention_q8", dict(
        shape=akv.shape(8, 2), B=2, q=P, q_pos=P, k_new=P, v_new=P, new_slot=P, kp=P, vp=P, k_scale=P, v_scale=P,
        S=10, kv_indptr=P, kv_indices=P, kv_pos=P, max_kv=50, out=P, ws=P, ws_bytes=1 << 30, stream=None), **change)


def _prefix(akv, **change):  # noqa: F811
    return _call(akv, "akv_prefix_attention", dict(
        shape=akv.shape(8, 2), G=1, group_indptr=P, max_rows=4, prefix_indptr=P, prefix_indices=P, max_prefix=50,
        B=2, q_indptr=P, n_rows=4, max_q=3, q=P, kp=P, vp=P, S=100, kv_indptr=P, kv_indices=P, max_kv=50, out=P,
        lse=P, ws=P, ws_bytes=1 << 30, stream=None), **change)


def test_append_refusals(akv):  # noqa: F811
    for change in (dict(n=-1), dict(S=-1), dict(k=None), dict(v=None), dict(slot=None), dict(kp=None),
                   dict(vp=None), dict(k_scale=None), dict(v_scale=None), dict(ks=120), dict(vs=127), dict(ks=132),
                   dict(k=P + 8), dict(v=P + 2), dict(kp=P + 8), dict(vp=P + 4), dict(k_scale=P + 2),
                   dict(v_scale=P + 8), dict(shape=akv.shape(7, 2))):
        assert _append(akv, **change) == INVALID, change
        assert akv.lib().akv_last_error()
    assert _append(akv, shape=akv.shape(8, 2, 128)) == UNSUPPORTED
    assert _append(akv, n=2 ** 30, shape=akv.shape(8, 2)) == UNSUPPORTED
    assert _append(akv, n=0, k=None, kp=None) == OK
    assert _append(akv, shape=akv.shape(8, 2, 64, "f32"), ks=130) == INVALID


def test_read_refusals(akv):  # noqa: F811
    for change in (dict(n=-1), dict(S=-1), dict(R=-1), dict(src=None), dict(k_out=None), dict(v_out=None),
                   dict(kp=None), dict(k_scale=None), dict(v_scale=None), dict(k_out=P + 8), dict(v_out=P + 4),
                   dict(vp=P + 8), dict(shape=akv.shape(7, 2))):
        assert _read(akv, **change) == INVALID, change
    assert _read(akv, n=0, src=None) == OK and _read(akv, R=0, k_out=None) == OK


def test_decode_refusals(akv):  # noqa: F811
    for change in (dict(B=-1), dict(max_kv=-1), dict(S=-1), dict(S=0), dict(q=None), dict(q_pos=None),
                   dict(kv_indptr=None), dict(kv_indices=None), dict(kv_pos=None), dict(out=None), dict(kp=None),
                   dict(k_scale=None), dict(k_new=None), dict(v_new=None), dict(new_slot=None),
                   dict(k_new=None, v_new=None), dict(q=P + 8), dict(out=P + 2), dict(k_new=P + 8), dict(kp=P + 8),
                   dict(shape=akv.shape(7, 2))):
        assert _decode(akv, **change) == INVALID, change
        assert akv.lib().akv_last_error()
    for change in (dict(B=65536), dict(max_kv=(1 << 30) + 1), dict(shape=akv.shape(8, 2, 128)),
                   dict(shape=akv.shape(65536, 1))):
        assert _decode(akv, **change) == UNSUPPORTED, change
    assert _decode(akv, B=0, q=None) == OK
    need = akv.akv_decode_q8_workspace(akv.shape(8, 2), 2, 50)
    assert need > 0
    for change in (dict(ws=None), dict(ws=P + 128), dict(ws_bytes=need - 1)):
        assert _decode(akv, **change) == WORKSPACE, change


def test_prefix_refusals(akv):  # noqa: F811
    for change in (dict(G=-1), dict(B=-1), dict(n_rows=-1), dict(max_rows=-1), dict(max_prefix=-1), dict(max_q=-1),
                   dict(max_kv=-1), dict(S=-1), dict(S=0), dict(group_indptr=None), dict(prefix_indptr=None),
                   dict(prefix_indices=None), dict(q_indptr=None), dict(kv_indptr=None), dict(kv_indices=None),
                   dict(q=None), dict(kp=None), dict(vp=None), dict(out=None), dict(q=P + 8), dict(kp=P + 2),
                   dict(out=P + 8), dict(shape=akv.shape(7, 2))):
        assert _prefix(akv, **change) == INVALID, change
        assert akv.lib().akv_last_error()
    for change in (dict(G=65536), dict(B=65536), dict(max_prefix=(1 << 30) + 1), dict(max_kv=(1 << 30) + 1),
                   dict(shape=akv.shape(8, 2, 128)),
                   dict(max_rows=2**31 - 1, n_rows=2**31 - 1, shape=akv.shape(4096, 1))):
        assert _prefix(akv, **change) == UNSUPPORTED, change
    for change in (dict(n_rows=0, q=None), dict(G=0, B=0, q=None)):
        assert _prefix(akv, **change) == OK, change
    need = akv.akv_prefix_workspace(akv.shape(8, 2), 1, 2, 4, 4, 50, 3, 50)
    assert need > 0
    for change in (dict(ws=None), dict(ws=P + 128), dict(ws_bytes=need - 1)):
        assert _prefix(akv, **change) == WORKSPACE, change


def test_workspace_queries_refuse_nonsense(akv):  # noqa: F811
    L, shp = akv.lib(), ctypes.byref(akv.shape(8, 2))
    assert L.akv_decode_q8_workspace(None, 1, 1) == 0
    for bad in ((0, 1), (1, -1), (1, (1 << 30) + 1)):
        assert L.akv_decode_q8_workspace(shp, *bad) == 0
    good = (1, 4, 50, 2, 4, 3, 50)
    assert L.akv_prefix_workspace(None, *good) == 0 and L.akv_prefix_workspace(shp, *good) > 0
    for i in range(7):
        assert L.akv_prefix_workspace(shp, *good[:i], -1, *good[i + 1:]) == 0


def test_workspaces_grow_with_their_bounds(akv):  # noqa: F811
    """The largest sizes that are allowed give sizes, no overflow."""
    for dtype in ("bf16", "f32"):
        shp = akv.shape(64, 8, 64, dtype)
        sizes = [akv.akv_decode_q8_workspace(shp, 14, n) for n in (1, 1000, 90000, 1 << 30)]
        assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))
        assert akv.akv_prefix_workspace(shp, 1, 14, 14, 14, 1 << 30, 1, 1 << 30) > 0


def test_the_tests_own_definition():
    """The 64-bit definition that the GPU tests compare with, by torch's conversion."""
    torch = pytest.importorskip("torch")
    assert np.array_equal(VALUES, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(),
                          equal_nan=True)
    x = np.random.default_rng(1).standard_normal((500, 64)) * np.exp(np.random.default_rng(2).normal(0, 9, (500, 1)))
    x = x.astype(np.float32).astype(np.float64)
    codes, byte = quantise(x)
    y = torch.from_numpy(x / 2.0 ** (byte[:, None] - 127.0)).float().to(torch.float8_e4m3fn)
    assert np.array_equal(codes, y.view(torch.uint8).numpy())
    top = np.abs(x).max(-1)
    assert np.all(top <= 448 * 2.0 ** (byte - 127.0)) and np.all(top > 448 * 2.0 ** (byte - 128.0))
    err = np.abs(held(codes, byte) - x)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (byte - 137.0)[:, None]))
