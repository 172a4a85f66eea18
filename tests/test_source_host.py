"""What the kernels' sources must not hold (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_drop_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_no_load_into_several_blocks(name):
    """The library's kernels run in replicas on any number of GPUs, and a load that
    one block multicasts into its cluster's shared memory is for runs on one GPU
    alone: no kernel issues one."""
    with open(os.path.join(CSRC, name)) as f:
        source = f.read()
    assert not re.search(r"multicast", source), name
