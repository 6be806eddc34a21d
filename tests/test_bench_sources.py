"""The recorded traffic stands for the sources that the benchmark measures: nothing that
its hash leaves out is part of them.  CPU only."""
import os
import re

import bench
from moe_grouped_gemm_block_amd import build

INCLUDE = re.compile(r'^\s*#\s*include\s*"([^"]+)"', re.M)


def included(name, seen=()):
    path = os.path.join(build.CSRC, name)
    if name in seen or not os.path.exists(path):
        return set(seen)
    seen = set(seen) | {name}
    for other in INCLUDE.findall(open(path).read()):
        seen = included(other, seen)
    return seen


def test_measured_sources_include_nothing_that_is_left_out():
    measured = [s for s in build.SOURCES if s not in bench.AROUND]
    assert "dg_api.hip" in measured and "kernels_e4m3.hip" in measured
    used = set()
    for s in measured:
        used |= included(s)
    assert "quant.hpp" in used and not used & bench.AROUND, used & bench.AROUND


def test_files_left_out_exist():
    assert all(os.path.exists(os.path.join(build.CSRC, f)) for f in bench.AROUND)
