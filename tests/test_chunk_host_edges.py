"""Host-side checks of the calls over a chunk of new tokens (no GPU): empty
buffers, which have no address, pass them.  Every call here is refused all the
same, for a later reason, so that nothing is enqueued."""
import pytest

from test_chunk_host import INVALID, P, _append, _evict, akv  # noqa: F401


def _reason(akv, status):  # noqa: F811
    assert status == INVALID
    return akv.lib().akv_last_error().decode()


@pytest.mark.parametrize("change", [
    dict(dropped=None, dropped_cap=0), dict(out_indices=None, out_pos=None, out_cap=0),
    dict(out_indices=None, kv_pos=None, out_pos=None, out_cap=0),
    dict(out_indices=None, out_pos=None, out_cap=0, dropped=None, dropped_cap=0)])
def test_evict_takes_empty_outputs(akv, change):  # noqa: F811
    assert "must not be mass" in _reason(akv, _evict(akv, out_mass=P, **change))
    # without the mass: the next reason is the positions'
    assert "together" in _reason(akv, _evict(akv, **{**change, "kv_pos": None, "out_pos": P, "out_mass": None,
                                                     "out_stride": 0}))


def test_append_takes_a_pool_without_slots(akv):  # noqa: F811
    why = _reason(akv, _append(akv, S=0, kp=None, vp=None, q_out=P, qs=1024))
    assert "in place" in why
