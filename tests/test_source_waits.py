"""Waits whose time is limited begin behind pdl_wait in their thread's own path: a kernel that starts early would otherwise count
the rest of the kernel in front of it, however long that runs."""
import re

import pytest

from test_source_loads import FILES, _code

LIMITED = re.compile(r"\b(?:mbar_wait_bounded|pair_wait(?:<true>)?)\s*\(")


def _kernels(code):
    for m in re.finditer(r"__global__[^{;]*?\bvoid\b[^{;]*?\b(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*\{", code):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[i], 0)
            i += 1
        yield m.group(1), code[m.end():i - 1]


def _roles(body):
    """The kernel's text in front of the split into roles, which begins at warp 0, and each role's."""
    start = re.search(r"\n  if \(warp == 0\) \{", body)
    if not start:
        return body, []
    parts = re.split(r"\n  \} else (?:if \([^{]*\) )?\{", body[start.end():])
    return body[:start.start()], parts


@pytest.mark.parametrize("name", FILES)
def test_limited_waits_come_behind_the_kernel_in_front(name):
    for kernel, body in _kernels(_code(name)):
        front, roles = _roles(body)
        for role in roles or [""]:
            path = front + role
            first = LIMITED.search(path)
            if first:
                assert "pdl_wait()" in path[:first.start()], kernel
