"""Host-only sizes of the sort (CPU): what dg_moe_sort refuses, the calls that
size its arguments refuse too, with the same status."""
import pytest

from moe_grouped_gemm_block_amd import dg

OK, INVALID, UNSUP = dg.DG_OK, dg.DG_ERR_INVALID_ARG, dg.DG_ERR_UNSUPPORTED
P = 1 << 20
BIG = 1 << 31


def sort(T, k, G, align, M):
    return dg.dg_moe_sort(P, dg.DG_IDX_I32, T, k, G, align, M, P, P, P, P, P, None)


@pytest.mark.parametrize("T,k,G,align,want", [
    (100, 2, 1025, 128, UNSUP), (100, 2, BIG - 1, 1, UNSUP), (1 << 29, 3, 8, 128, UNSUP), (1 << 30, 2, 8, 1, INVALID),
    (BIG, 1, 8, 1, INVALID), (1 << 30, BIG - 1, 8, 1, INVALID), (-1, 2, 8, 1, INVALID), (100, 0, 8, 1, INVALID),
    (100, 2, 0, 1, INVALID), (100, 2, -5, 128, INVALID),
])
def test_sizes_refuse_what_the_sort_refuses(T, k, G, align, want):
    assert sort(T, k, G, align, BIG - 128) == want
    assert dg.dg_moe_rows(T, k, G, align) == want
    assert dg.dg_moe_sort_workspace(T, k, G) == want


def test_the_largest_sizes_are_given():
    assert dg.dg_moe_rows(1 << 30, 1, 1024, 128) == ((1 << 30) + 127 * 1024) // 128 * 128
    assert dg.dg_moe_sort_workspace(1 << 30, 1, 1024) > 0
