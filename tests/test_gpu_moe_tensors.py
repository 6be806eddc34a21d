"""What the mixture-of-experts operators' output tensors are to torch: saved,
loaded, kept and written as any other tensor.  Needs a GPU."""
import io

import pytest
import torch

from moe_grouped_gemm_block_amd import dg

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def saved_and_loaded(value):
    f = io.BytesIO()
    torch.save(value, f)
    f.seek(0)
    return torch.load(f, weights_only=True, map_location=DEV)


@pytest.mark.parametrize("M,I", [(3, 16), (130, 272), (0, 128)])
def test_codes_and_scales_are_saved_and_loaded(M, I):
    """A checkpoint, or a quantised operand, in one file."""
    h = torch.randn(M, 2 * I, device=DEV)
    ids = torch.randint(0, 4, (M, 2), device=DEV)
    plan = dg.moe_sort(ids, 4)
    for outputs in (dg.swiglu_fp8(h), dg.moe_permute_fp8(h, plan.slot_row, plan.row_slot)):
        back = saved_and_loaded(outputs)
        for a, b in zip(outputs, back):
            assert a.dtype == b.dtype and torch.equal(a, b)
        for codes in outputs[::2]:
            assert codes.untyped_storage().nbytes() == codes.numel()      # nothing beside them
    assert all(torch.equal(a, b) for a, b in zip(plan, saved_and_loaded(tuple(plan))))


@pytest.mark.parametrize("T,k,G", [(100, 2, 64), (10000, 4, 256)])
def test_a_plan_keeps_no_workspace(T, k, G):
    """The sort of more than 8192 slots has a workspace, which ends with the call."""
    plan = dg.moe_sort(torch.randint(0, G, (T, k), device=DEV), G)
    assert (dg.dg_moe_sort_workspace(T, k, G) > 0) == (T * k > 8192)
    held = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in plan}
    assert sum(held.values()) == sum(4 * t.numel() for t in plan)
