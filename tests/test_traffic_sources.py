"""The recorded DRAM traffic of a plan path is tied to its kernels' sources: every header of this library that they
include, directly or through another, is among the files whose hash is compared."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "block_scaled_mxfp4_bf16_gb300", "csrc")


def _included(name: str, seen: set) -> set:
    with open(os.path.join(CSRC, name)) as f:
        for header in re.findall(r'^\s*#include "([^"]+)"', f.read(), re.M):
            if os.path.exists(os.path.join(CSRC, header)) and header not in seen:
                seen.add(header)
                _included(header, seen)
    return seen


@pytest.mark.parametrize("path", bench.KERNEL_SOURCES)
def test_every_included_header_is_hashed(path):
    listed = bench.KERNEL_SOURCES[path]
    for unit in (n for n in listed if n.endswith(".cu")):
        found = {n for n in _included(unit, set()) if not n.startswith("..")}
        assert found, unit
        assert found <= set(listed), (unit, sorted(found - set(listed)))
