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


def test_written_outputs_change_their_version():
    """A tensor that an operator writes counts as written: autograd refuses to
    use it where an earlier operation saved what it held."""
    T, k, G, H = 40, 2, 4, 128
    x = torch.randn(T, H, device=DEV).bfloat16()
    plan = dg.moe_sort(torch.randint(0, G, (T, k), device=DEV), G)
    M = plan.row_slot.numel()
    w = torch.rand(T, k, device=DEV)
    new = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device=DEV)
    Q, S = new(M, H, dtype=torch.uint8), new(M, 1, dtype=torch.float32)
    A, sA, Hq, sH = dg.swiglu_fp8(torch.randn(M, 2 * H, device=DEV))
    calls = {
        "moe_permute": lambda o: dg.moe_permute(x, plan.slot_row, plan.row_slot, Y=o[0]),
        "moe_permute_fp8": lambda o: dg.moe_permute_fp8(x, plan.slot_row, plan.row_slot, Q=o[0], S=o[1]),
        "moe_combine": lambda o: dg.moe_combine(new(M, H), plan.slot_row, w, out=o[0]),
        "moe_combine_bwd": lambda o: dg.moe_combine_bwd(x, new(M, H), plan.slot_row, plan.row_slot, w, dY=o[0],
                                                        dweights=o[1]),
        "swiglu_fp8_bwd": lambda o: dg.swiglu_fp8_bwd(new(M, H), Hq, sH, dH=o[0]),
        "grouped_wgrad_fp8": lambda o: dg.grouped_wgrad_fp8(new(M, H), A, sA, plan.group_offsets, dW=o[0],
                                                            accumulate=True),
    }
    outputs = {"moe_permute": [new(M, H)], "moe_permute_fp8": [Q, S], "moe_combine": [new(T, H)],
               "moe_combine_bwd": [new(M, H), new(T, k, dtype=torch.float32)], "swiglu_fp8_bwd": [new(M, 2 * H)],
               "grouped_wgrad_fp8": [new(G, H, H, dtype=torch.float32)]}
    for name, call in calls.items():
        before = [t._version for t in outputs[name]]
        call(outputs[name])
        assert all(t._version > v for t, v in zip(outputs[name], before)), name
    leaf = torch.ones(G, H, H, device=DEV, requires_grad=True)
    dw = outputs["grouped_wgrad_fp8"][0]
    loss = (leaf * dw).sum()
    calls["grouped_wgrad_fp8"]([dw])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():                               # tensors without a version
        out = new(T, H)
        dg.moe_combine(new(M, H), plan.slot_row, w, out=out)


@pytest.mark.parametrize("args,status", [((1025,), dg.DG_ERR_UNSUPPORTED), ((2 ** 31 - 1,), dg.DG_ERR_UNSUPPORTED),
                                         ((0,), dg.DG_ERR_INVALID_ARG), ((8, 64), dg.DG_ERR_INVALID_ARG),
                                         ((8, 128, 128), dg.DG_ERR_INVALID_ARG),
                                         ((8, 128, 2 ** 31 - 2 ** 20 + 1), dg.DG_ERR_INVALID_ARG),
                                         ((8, 1, 2 ** 31), dg.DG_ERR_INVALID_ARG)])
def test_a_refused_sort_allocates_nothing(args, status):
    ids = torch.zeros(100, 2, dtype=torch.int32, device=DEV)
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(dg.DGError) as e:
        dg.moe_sort(ids, *args)
    assert e.value.status == status
    assert torch.cuda.max_memory_allocated() == before
