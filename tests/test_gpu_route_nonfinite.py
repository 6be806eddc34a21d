"""NaN and infinite logits in the router with a bias.  Needs a GPU."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from test_gpu_route import DEV, INF, check, logits, n

pytestmark = pytest.mark.gpu

NAN = float("nan")
# (rows of 16 lanes and waves, one and several values a lane)
SHAPES = [(40, 12, 4), (40, 200, 8), (4100, 200, 8), (40, 600, 8)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("renorm", [True, False])
def test_rows_without_numbers_have_no_weights(T, E, k, value, renorm):
    """Under softmax one NaN or +inf leaves a token no scores: all its weights are NaN,
    also where the experts that are chosen have finite logits."""
    x = logits(T, E, torch.float32, 9)
    x[3, E - 1] = value
    bias = torch.zeros(E, device=DEV)
    r = dg.moe_route(x.to(DEV), k, renormalise=renorm, bias=bias)
    assert np.isnan(n(r.weights)[3]).all() and n(r.ids)[3].min() >= 0 and len(set(n(r.ids)[3].tolist())) == k
    rows = [t for t in range(T) if t != 3]
    assert np.isfinite(n(r.weights)[rows]).all()


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("kind", ["plain", "equal"])
def test_a_bias_closes_experts_whose_logits_are_no_numbers(T, E, k, score, value, kind):
    x = logits(T, E, torch.float32, 9, kind)
    x[::3, E - 2] = value
    x[5, E - 4:] = NAN
    bias = torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.1
    bias[E - 4:] = -INF
    r = dg.moe_route(x.to(DEV), k, score=score, bias=bias.to(DEV), balance=False)
    ids = n(r.ids)
    assert ids.min() >= 0 and ids.max() < E - 4 and all(len(set(row)) == k for row in ids.tolist())
    if score == "sigmoid":                        # the open experts' scores do not know of them
        x[:, E - 4:] = -INF
        want, _ = check(x, k, score, True, bias=bias, balance=False)
        assert torch.equal(r.ids, want.ids) and torch.equal(r.weights, want.weights)


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_without_a_choice_add_nothing_to_the_load(T, E, k, score):
    """Tokens whose experts a bias has closed, all of them, whatever their logits are."""
    x = logits(T, E, torch.float32, 9)
    bias = torch.zeros(E)
    bias[E - 3:] = -INF
    x[7, : E - 3] = -INF
    x[9, : E - 3] = -INF
    want, _ = check(x, k, score, True, bias=bias)
    assert int(want.routed) == T - 2
    x[7, E - 1], x[9, E - 2], x[9, E - 1] = NAN, INF, NAN
    got = dg.moe_route(x.to(DEV), k, score=score, bias=bias.to(DEV))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
