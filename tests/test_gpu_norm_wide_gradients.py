"""The norms' gradients of rows that go through memory, against the float64 oracle: FP32
rows of odd widths above 4096 columns, and rows above 8192 of which a workgroup takes
several, so that it adds to its own column sums.  Needs a GPU.

Tolerances are those of test_gpu_norm.py, whose check this is."""
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from test_gpu_norm import B, F, check, check_bwd, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


@pytest.mark.parametrize("T,H", [(3, 4097), (520, 4097), (520, 5001), (520, 8191)])
@pytest.mark.parametrize("rt,dt", [(F, F), (F, B), (B, F), (B, B)])
def test_odd_widths_past_4096(T, H, rt, dt):
    p = problem(T, H, rt, dt, gate="channel")
    p["R"][T // 2] *= 1e-18                       # (with this eps the sums of one row are in 64 bits)
    check_bwd(p, alpha=0.5, eps=1e-8)
    check_bwd(problem(T, H, rt, dt, gate="token"), with_dR=False)
    check(p, alpha=0.5, eps=1e-8)


@pytest.mark.parametrize("T,H", [(1100, 9000), (1100, 8193), (700, 20000)])
@pytest.mark.parametrize("rt,dt", [(B, B), (F, F)])
def test_wide_rows_several_a_workgroup(T, H, rt, dt):
    """(At most 2^22 / H workgroups: two to four rows each.)"""
    check_bwd(problem(T, H, rt, dt, gate="channel"), alpha=0.5)
