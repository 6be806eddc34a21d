"""The single-stage build's weight gradient: libdg_stages1.so copies a step's
rows only after the previous step's have been used and waits for all of them,
where libdg.so counts the copies in flight.  The arithmetic and its order are the
same, so the two must give identical bytes; a difference would point at a copy
that is read before it has landed or overwritten before it is read.  Each library
runs in a child process (tests/wgrad_stages_child.py).  Needs a GPU."""
import os
import subprocess
import sys

import numpy as np
import pytest

from moe_grouped_gemm_block_amd import build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def run_child(lib, out):
    r = subprocess.run([sys.executable, os.path.join(HERE, "wgrad_stages_child.py"), out],
                       env=dict(os.environ, DG_LIBRARY=lib), capture_output=True, text=True, timeout=100)
    print(r.stdout, file=sys.stderr)
    assert r.returncode == 0, r.stdout + r.stderr[-2000:]


def test_single_stage_weight_gradient_gives_identical_bytes(tmp_path):
    assert os.path.exists(build.LIB_STAGES1), "libdg_stages1.so is not built"
    a, b = str(tmp_path / "ahead.npz"), str(tmp_path / "one.npz")
    run_child(build.LIB, a)
    run_child(build.LIB_STAGES1, b)
    A, B = np.load(a), np.load(b)
    assert sorted(A.files) == sorted(B.files) and len(A.files) > 0
    for k in A.files:
        assert A[k].any() and np.array_equal(A[k], B[k]), f"{k}: single-stage output differs"
