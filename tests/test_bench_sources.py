"""The source files that key a kernel's counted traffic in bench.py hold everything the kernel is compiled from (no GPU)."""
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

LAUNCHERS = "sp24_launch.h"  # host declarations, which kernels do not see


def included(name):
    found = {name}
    for header in re.findall(r'#include "(\w+\.h)"', open(os.path.join(bench.CSRC, name)).read()):
        if header != LAUNCHERS:
            found |= included(header)
    return found


def source_lists():
    lists = re.findall(r'\(("\w+\.(?:hip|h)"(?:, "\w+\.(?:hip|h)")+)\)', open(os.path.join(ROOT, "bench.py")).read())
    return sorted({tuple(re.findall(r'"([^"]+)"', x)) for x in lists} | {bench.gemm_sources(n) for n in (1, 16, 64, 65, 4096)})


@pytest.mark.parametrize("files", source_lists(), ids=lambda f: f[0])
def test_headers_of_the_kernels_are_listed(files):
    missing = set().union(*(included(f) for f in files)) - set(files)
    assert not missing, missing


def test_every_list_was_found():
    assert len(source_lists()) >= 5 and any("norms.hip" in f for f in source_lists())
