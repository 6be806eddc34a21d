"""A library of an earlier build, named by DG_LIBRARY, keeps working for what it
has (CPU: a stand-in of empty functions, loaded in a child process)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PRODUCTS = ("dg_gemm_fp8_blockscaled", "dg_grouped_gemm_fp8", "dg_gemm_fp8_ex", "dg_gemm_fp8_ex_noalloc",
            "dg_grouped_gemm_fp8_ex", "dg_grouped_gemm_fp8_ex_counts", "dg_grouped_gemm_fp8_segments",
            "dg_quantize_fp8_blockscaled")

CHILD = """
from moe_grouped_gemm_block_amd import dg
assert dg.dg_gemm_fp8_blockscaled(1, 2, 3, 4, 5, 6, 7, 8, 0, None) == 7
assert dg.dg_quantize_fp8_blockscaled(1, 0, 2, 3, 4, 5, 128, None) == 7
assert dg.dg_status_string(0) == "stand-in"
for call in (lambda: dg.dg_moe_rows(1, 1, 1, 1), lambda: dg.dg_swiglu_fp8_bwd(1, 1, 1, 1, 1, 1, 1, None)):
    try:
        call()
    except AttributeError as e:
        assert "dg_" in str(e), e
    else:
        raise SystemExit("a function that the library lacks was called")
try:
    dg.binding()
except RuntimeError as e:
    assert "build" in str(e), e
else:
    raise SystemExit("the binding took a library that lacks its functions")
print("fine")
"""


def test_what_an_older_library_has_still_works(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, so = str(tmp_path / "old.c"), str(tmp_path / "libold.so")
    with open(src, "w") as f:
        f.write("".join(f"int {n}(void) {{ return 7; }}\n" for n in PRODUCTS))
        f.write('const char* dg_status_string(int s) { return "stand-in"; }\n')
    subprocess.run([cc, "-shared", "-fPIC", src, "-o", so], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD], env=dict(os.environ, DG_LIBRARY=so, PYTHONPATH=ROOT),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr[-2000:]
