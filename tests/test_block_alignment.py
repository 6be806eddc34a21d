"""Alignment that the router and the norms ask for where rows are not of whole vectors
(CPU only): every call below is refused before any HIP call; the fake addresses are
never dereferenced."""
import pytest

from moe_grouped_gemm_block_amd import dg
from test_block_abi import INVALID, NORM, NORM_BWD, P, ROUTE, ROUTE_BWD, call


@pytest.mark.parametrize("kw", [dict(E=63, x=P + 2), dict(E=63, dt=1, x=P + 1), dict(dt=1, x=P + 4), dict(dt=1, x=P + 2)])
def test_route(kw):
    assert call(dg.dg_moe_route, ROUTE, kw) == INVALID
    assert call(dg.dg_moe_route_bwd, ROUTE_BWD, kw) == INVALID
    assert call(dg.dg_moe_route_bwd, ROUTE_BWD, dict(kw, x=P, dx=kw["x"])) == INVALID


@pytest.mark.parametrize("kw", [dict(R=P + 1), dict(Y=2 * P + 1), dict(rt=0, R=P + 2), dict(dt=0, Y=2 * P + 2), dict(w_post=P + 2),
                                dict(gate=P + 2), dict(gate=P + 1, kind=2), dict(w_pre=P + 1)])
def test_norm(kw):
    assert call(dg.dg_residual_norm, NORM, dict(kw, H=257, Q=None, S=None)) == INVALID
    assert call(dg.dg_residual_norm_bwd, NORM_BWD, dict(kw, H=257)) == INVALID


def test_norm_outputs():
    for kw in (dict(Ro=3 * P + 1), dict(N=4 * P + 1), dict(rt=0, Ro=3 * P + 2), dict(dt=0, N=4 * P + 2)):
        assert call(dg.dg_residual_norm, NORM, dict(kw, H=257, Q=None, S=None)) == INVALID
    for kw in (dict(dRo=3 * P + 1), dict(dY=4 * P + 1), dict(dR=5 * P + 1), dict(dN=6 * P + 1), dict(rt=0, dR=5 * P + 2),
               dict(dt=0, dN=6 * P + 2)):
        assert call(dg.dg_residual_norm_bwd, NORM_BWD, dict(kw, H=257)) == INVALID
