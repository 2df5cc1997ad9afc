"""A question how many blocks or clusters of a kernel fit on the device counts its dynamic shared memory only within the
allowance that the kernel has at that moment: every function that asks raises the allowance first."""
import os
import re

import pytest

from test_source_loads import CSRC, FILES, _code

ASKS = re.compile(r"cudaOccupancyMax\w+\s*\(")


def _functions_that_ask(code):
    """Bodies of the functions that ask, up to the question."""
    for m in ASKS.finditer(code):
        depth, i = 0, m.start()
        while i > 0:                    # back to the brace that opens the outermost block below a namespace
            i -= 1
            if code[i] == "}":
                depth += 1
            elif code[i] == "{":
                if depth == 0 and re.search(r"\)\s*$", code[:i]) and not re.search(r"\b(?:if|for|while|switch)\s*\([^{}]*\)\s*$", code[:i]):
                    break
                depth = max(depth - 1, 0)
        yield code[i:m.start()]


@pytest.mark.parametrize("name", FILES)
def test_allowance_before_the_question(name):
    for body in _functions_that_ask(_code(name)):
        assert re.search(r"allow_smem\s*\(|cudaFuncAttributeMaxDynamicSharedMemorySize", body), (name, body)


def test_there_are_such_questions():
    assert sum(len(ASKS.findall(_code(f))) for f in os.listdir(CSRC) if f in FILES) >= 2
