"""A call's first kernel starts after the caller's last one has ended and its
writes are seen: no programmatic edge leaves the caller's kernel in a captured
graph.  Only a call's own kernels follow one another by such edges."""
import ctypes

import numpy as np
import pytest

import kv_cache_drop_gb300 as akv
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu


class _Edge(ctypes.Structure):  # CUgraphEdgeData
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def _edges(fn):
    """(from, to, programmatic) of the graph that fn(stream) leaves behind a kernel of
    the caller's; the caller's kernel is the one node without an incoming edge."""
    import torch
    cuda = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    x = torch.zeros(1000, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.add(x, 1, out=x)  # loaded
        stream.synchronize()
        assert cuda.cuStreamBeginCapture_v2(ctypes.c_void_p(stream.cuda_stream), 2) == 0
        try:
            torch.add(x, 1, out=x)
            fn(stream)
        finally:
            graph = ctypes.c_void_p()
            rc = cuda.cuStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph))
    assert rc == 0
    n = ctypes.c_size_t(0)
    assert cuda.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)) == 0
    a, b, e = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (_Edge * n.value)()
    assert cuda.cuGraphGetEdges_v2(graph, a, b, e, ctypes.byref(n)) == 0
    cuda.cuGraphDestroy(graph)
    return [(a[i], b[i], e[i].type == 1) for i in range(n.value)]


CASES = {  # rows, own lists, groups' first requests, prefixes
    "both passes": ([1, 2], [200, 150], [0, 2], [700]),
    "prefix only": ([1, 2], [0, 0], [0, 2], [700]),
    "own lists only": ([1, 2], [200, 150], [0, 2], [0]),
    "no list": ([1, 2], [0, 0], [0, 2], [0]),
    "no list, many rows": ([300, 2], [0, 0], [0, 2], [0]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_prefix_call_follows_the_caller(name, dtype):
    m, n, cut, p = CASES[name]
    bt = Batch(3, m, n, cut, p, 16, 4, dtype)
    d = bt.device()
    out, lse = bt.run(d)  # loads the kernels
    bt.check(out, lse)
    ws = bt.workspace()

    def call(stream):
        akv.akv_prefix_attention(bt.shp, bt.G, d["g_ptr"], d["pre_ptr"], d["pre"], bt.B, d["q_ptr"], d["q"], d["k"],
                                 d["v"], d["kv_ptr"], d["idx"], out=out, lse=lse, workspace=ws, stream=stream,
                                 **bt.sizes)

    edges = _edges(call)
    passes = (max(n) > 0) + (max(p) > 0)
    assert len(edges) == 1 + passes
    caller = {a for a, _, _ in edges} - {b for _, b, _ in edges}
    assert len(caller) == 1
    assert [late for a, _, late in edges if a in caller] == [False]
    assert all(late for a, _, late in edges if a not in caller)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_limits_written_by_the_kernel_before(dtype):
    """A call without lists takes the rows that the kernel before it wrote."""
    import torch
    rows, Hq, Hkv = 4000, 16, 4
    shp = akv.shape(Hq, Hkv, 64, dtype)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = torch.ones(rows, Hq, 64, dtype=dt, device="cuda")
    pool, none = torch.ones(4, Hkv, 64, dtype=dt, device="cuda"), akv.i32_device([])
    lists, want = akv.i32_device([0, 0]), akv.i32_device([0, 0])
    ws = torch.zeros(akv.akv_prefix_workspace(shp, 1, 1, rows, rows, 0, rows, 0), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    for _ in range(20):
        end = int(rng.integers(1, rows))
        limit = akv.i32_device([0, end])
        out, lse = torch.full_like(q, 7.0), torch.full((rows, Hq), 7.0, device="cuda")
        torch.add(limit, 0, out=want)
        akv.akv_prefix_attention(shp, 1, want, lists, none, 1, want, q, pool, pool, lists, none, max_rows=rows,
                                 max_prefix=0, max_q=rows, max_kv=0, out=out, lse=lse, workspace=ws)
        assert not out[:end].any() and bool((out[end:] == 7).all())
        assert bool(torch.isneginf(lse[:end]).all()) and bool((lse[end:] == 7).all())
