"""Kernels are launched while the one before them on the stream still runs (launch_pdl) and wait for it on the device, so
memory that it writes is written during their own lifetime: they read with ordinary loads.  The read-only path (__ldg, the
.nc form of a load, parameters that are const and __restrict__) is only defined for memory that nothing writes meanwhile."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_layer_routing_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h")))
# Bias rows and a saved act(gate), which no kernel of the library writes: whatever did is complete before the kernels in
# front of these GEMMs let them start.
CALLERS_OWN = {"gemm_kernel.cuh": 2, "gemm_pair_kernel.cuh": 1}


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"/\*.*?\*/|//[^\n]*", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    assert len(re.findall(r"__ldg\s*\(|\bld\.global(?:\.\w+)*\.nc\b", _code(name))) == CALLERS_OWN.get(name, 0)


@pytest.mark.parametrize("name", FILES)
def test_parameters_of_kernels_that_start_early(name):
    """Kernels that plain launches start (<<< >>>) begin after everything before them and may keep the qualifier."""
    code = _code(name)
    plain = set(re.findall(r"\b(\w+)\s*(?:<[^<>;]*>)?\s*<<<", code))
    early = set(re.findall(r"launch_pdl\(\s*(\w+)", code))
    kernels = re.findall(r"__global__[^{;]*?\bvoid\b[^{;]*?\b(\w+)\s*\(((?:[^()]|\([^()]*\))*)\)\s*\{", code)
    for kernel, parameters in kernels:
        if kernel in plain:
            assert kernel not in early, kernel
        else:
            assert not re.search(r"\bconst\b[^,]*__restrict__", parameters), kernel
