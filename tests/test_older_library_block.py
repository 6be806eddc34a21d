"""A library of an earlier build that has the mixture-of-experts operators but not those
around a block keeps working for what it has (CPU: a stand-in of empty functions, loaded
in a child process)."""
import os
import shutil
import subprocess
import sys

import pytest

from moe_grouped_gemm_block_amd import dg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NEW = ("dg_moe_route", "dg_moe_route_workspace", "dg_moe_route_bwd", "dg_residual_norm", "dg_residual_norm_bwd",
       "dg_residual_norm_bwd_workspace", "dg_grad_norm", "dg_grad_norm_workspace", "dg_clip_grads")

CHILD = """
import torch
from moe_grouped_gemm_block_amd import dg
x, i = torch.zeros(2, 8), torch.zeros(2, 1, dtype=torch.int32)
assert dg.dg_moe_rows(1, 1, 1, 1) == 7
dg.binding()
try:
    dg.moe_permute(x, i, i[:, 0])
except ValueError as e:
    assert "device tensor" in str(e), e
for call in (lambda: dg.moe_route(x, 1), lambda: dg.moe_route_bwd(x, x, i), lambda: dg.residual_norm(x, w_pre=x[0]),
             lambda: dg.residual_norm_bwd(x, x, x, w_pre=x[0]), lambda: dg.grad_norm([x]),
             lambda: dg.clip_grads([x], x, 1.0)):
    try:
        call()
    except RuntimeError as e:
        assert "lacks dg_" in str(e) and "build" in str(e), e
    else:
        raise SystemExit("a function that the library lacks was called")
print("fine")
"""


def test_what_an_older_library_has_still_works(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    if not os.path.exists(os.path.join(ROOT, "moe_grouped_gemm_block_amd", "_dg_torch.so")):
        pytest.skip("the binding is not built")
    src, so = str(tmp_path / "old.c"), str(tmp_path / "libold.so")
    with open(src, "w") as f:
        f.write("".join(f"long {name}(void) {{ return 7; }}\n" for name in dg.EXPORTED
                        if name not in NEW and name != "dg_status_string"))
        f.write('const char* dg_status_string(int s) { return "stand-in"; }\n')
    subprocess.run([cc, "-shared", "-fPIC", src, "-o", so], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD], env=dict(os.environ, DG_LIBRARY=so, PYTHONPATH=ROOT),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr[-2000:]
