"""Kernels are launched while the one before them on the stream still runs and wait for it on the device, so memory that
it writes is written during their own lifetime: they read with ordinary loads.  The read-only path (__ldg, the .nc form of
a load, parameters that are const and __restrict__) is only defined for memory that nothing writes meanwhile."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_layer_routing_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|\bld\.global(\.\w+)*\.nc\b|\bconst\s+\w+\s*\*\s*__restrict__")
FILES = ["layer_norm.cu", "balance.cu", "ckpt8.cu"]


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"/\*.*?\*/|//[^\n]*", "", f.read(), flags=re.S)
    assert not [m.group(0) for m in READ_ONLY.finditer(code)]
