"""The router's kernels for large batches against the float64 oracle: 65 to 256 experts
of more than 4096 tokens go over rows of 16 lanes, and loads of more than 16384 partial
sums are added up by several workgroups.  Needs a GPU.

Tolerances are those of test_gpu_route.py, whose checks these are."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import block as O
from test_gpu_route import INF, check, check_bwd, logits, n

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def some_bias(E, seed=5):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 0.1


@pytest.mark.parametrize("T", [4096, 4097, 4163])
@pytest.mark.parametrize("E,k", [(65, 3), (128, 8), (255, 16), (256, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(T, E, k, dtype, score):
    x = logits(T, E, dtype, seed=T + E)
    check(x, k, score, renorm=True, scale=2.5)
    if T == 4097:
        check(x, k, score, renorm=False, bias=some_bias(E))
        check(x, k, score, renorm=False, balance=False)


@pytest.mark.parametrize("kind", ["closed", "ties", "equal", "far", "lowest"])
@pytest.mark.parametrize("E,k", [(100, 8), (253, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_hard_rows(kind, E, k, score):
    """Of rows of 16 lanes, with and without a bias."""
    bias = some_bias(E)
    bias[::7] = -INF
    for dtype in (torch.float32, torch.bfloat16):
        x = logits(4101, E, dtype, 3, kind)
        check(x, k, score, True)
        check(x, k, score, False, bias=bias)


@pytest.mark.parametrize("T,E,k", [(6000, 256, 8), (4096, 256, 8), (600, 1000, 8), (5000, 1024, 4), (9000, 200, 2)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_loads_of_several_workgroups(T, E, k, biased):
    """More partial sums than one workgroup adds up, of both kinds of lanes, some rows without a token."""
    mask = torch.rand(T, generator=torch.Generator().manual_seed(8)) < 0.9
    bias = some_bias(E) if biased else None
    a, _ = check(logits(T, E, torch.float32, 6), k, "sigmoid", True, bias=bias, mask=mask)
    b, _ = check(logits(T, E, torch.float32, 6), k, "sigmoid", True, bias=bias, mask=mask)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("T", [4096, 4097])
@pytest.mark.parametrize("E,k", [(65, 3), (128, 8), (255, 16), (256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bwd(T, E, k, score):
    for dtype in (torch.float32, torch.bfloat16):
        x = logits(T, E, dtype, T + E)
        ids = O.choose(n(x), k, False)
        for renorm in (True, False):
            check_bwd(x, ids, score, renorm, loss=renorm or T == 4097)


@pytest.mark.parametrize("kind", ["closed", "equal", "far", "lowest"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bwd_hard_rows(kind, score):
    for renorm in (True, False):
        x = logits(4101, 253, torch.bfloat16, 3, kind)
        ids = O.choose(n(x), 6, False, mask=np.arange(4101) % 7 != 0)
        ids[5] = 9                                            # an expert named six times
        check_bwd(x, ids, score, renorm, True)
