"""The 8-bit cache where it can go wrong: a workspace sized for larger calls."""
import pytest

import kv_cache_drop_gb300 as akv
from test_gpu_kv8 import Batch

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
