"""Clipping of gradients whose norm is far above the limit.  Needs a GPU.

The tolerance is test_gpu_clip.py's, whose check this is: the factor max_norm / norm
rounds once, 2^-24 of itself, also where FP32's normal numbers do not hold it."""
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from test_gpu_clip import B, F, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


@pytest.mark.parametrize("size,max_norm", [(1e36, 1.0), (1e36, 1e-3), (1e36, 1e-7), (3e35, 1e-30)])
@pytest.mark.parametrize("kind", [F, B])
@pytest.mark.parametrize("place", ["in place", "f32", "bf16"])
def test_clip_far_above_the_limit(size, max_norm, kind, place):
    grads = make([(300,), (7, 11), (1001,)], [kind] * 3, size=size)
    out = None
    if place != "in place":
        out = [torch.empty_like(t, dtype={"f32": F, "bf16": B}[place]) for t in grads]
    check(grads, max_norm, out)
