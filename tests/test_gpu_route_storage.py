"""What the router's results keep in memory.  Needs a GPU."""
import io

import pytest
import torch

from moe_grouped_gemm_block_amd import dg

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("T,E,k", [(1, 64, 2), (700, 64, 2), (700, 256, 8), (5000, 60, 6)])
@pytest.mark.parametrize("balance", [True, False])
def test_results_of_tokens_lie_alone(T, E, k, balance):
    """A loss that is kept keeps none of its batch, and ids and weights are aligned as
    tensors of their own are."""
    r = dg.moe_route(torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)), k, balance=balance)
    for t in (r.ids, r.weights):
        assert t.untyped_storage().nbytes() == 4 * T * k and t.data_ptr() % 256 == 0
    if balance:
        for t in (r.counts, r.prob_sums, r.routed, r.loss):
            assert t.untyped_storage().nbytes() == 4 * (E + 1)
        f = io.BytesIO()
        torch.save(r._asdict(), f)
        f.seek(0)
        for name, t in torch.load(f, weights_only=True).items():
            assert torch.equal(t, getattr(r, name)), name
