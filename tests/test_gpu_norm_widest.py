"""The norms of the widest rows that they take, and of rows just past it.  Needs a GPU.

Tolerances are those of test_gpu_norm.py, whose checks these are."""
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from test_gpu_norm import B, DEV, F, check, check_bwd, problem

pytestmark = pytest.mark.gpu

WIDEST = 1 << 22


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


@pytest.mark.parametrize("T,H,rt,dt", [(3, WIDEST, B, B), (2, WIDEST - 1, F, B), (3, WIDEST - 3, B, B)])
def test_widest_rows(T, H, rt, dt):
    p = problem(T, H, rt, dt, gate="channel")
    check(p, alpha=0.5, codes="pow2" if H % 16 == 0 else None)
    check_bwd(p, alpha=0.5)


def test_wider_rows_are_refused():
    x, w = torch.zeros(1, WIDEST + 1, device=DEV), torch.ones(WIDEST + 1, device=DEV)
    for bad in (lambda: dg.residual_norm(x, w_pre=w), lambda: dg.residual_norm_bwd(x, x, x, w_pre=w)):
        with pytest.raises(dg.DGError):
            bad()
