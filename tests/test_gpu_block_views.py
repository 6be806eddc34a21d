"""Operands of the norms and the router that lie at any element of a larger tensor: rows
that are not of whole vectors are read and written there.  Needs a GPU."""
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from test_gpu_norm import B, DEV, F, dev, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def moved(t, at):
    """The same values `at` elements into a larger tensor of NaN."""
    if t is None or t.numel() == 0:
        return t
    fill = float("nan") if t.is_floating_point() else 99
    whole = torch.full((t.numel() + at + 9,), fill, dtype=t.dtype, device=t.device)
    out = whole[at:at + t.numel()].view(t.shape)
    out.copy_(t)
    return out


def same(a, b):
    for p, q in zip(a, b):
        assert (p is None) == (q is None) and (p is None or torch.equal(p, q))


@pytest.mark.parametrize("T,H", [(1, 1), (5, 7), (40, 513), (600, 1423), (3, 4097), (2, 8193), (3, 9001)])
@pytest.mark.parametrize("rt,dt", [(B, B), (F, F), (F, B), (B, F)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_norm(T, H, rt, dt, gate):
    p = {k: dev(v) for k, v in problem(T, H, rt, dt, gate=gate).items()}
    g = torch.Generator(device=DEV).manual_seed(4)
    dR, dN = (torch.randn(T, H, device=DEV, generator=g).to(t) for t in (rt, dt))

    def calls(p, dR, dN):
        kw = dict(w_post=p["w_post"], gate=p["gate"], alpha=0.5, w_pre=p["w_pre"])
        o = dg.residual_norm(p["R"], p["Y"], **kw)
        return (*o, *dg.residual_norm_bwd(dR, dN, p["R"], p["Y"], **kw),
                *dg.residual_norm(p["R"], w_pre=p["w_pre"], dtype="f32"))

    want = calls(p, dR, dN)
    for at in range(1, 9):
        same(calls({k: moved(v, at if k != "Y" else 9 - at) for k, v in p.items()}, moved(dR, at), moved(dN, 9 - at)), want)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (40, 7, 3), (40, 62, 4), (300, 255, 8), (4100, 255, 8), (30, 999, 8)])
@pytest.mark.parametrize("dtype", [F, B])
def test_route(T, E, k, dtype):
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(T, E, device=DEV, generator=g).to(dtype)
    dw, bias = torch.randn(T, k, device=DEV, generator=g), torch.randn(E, device=DEV, generator=g) * 0.1

    def calls(x, dw, bias, out):
        r = dg.moe_route(x, k, score="sigmoid", bias=bias)
        dx = dg.moe_route_bwd(dw, x, r.ids, score="sigmoid", dloss=r.loss, counts=r.counts, routed=r.routed, dlogits=out)
        return (*r, dx)

    want = calls(x, dw, bias, None)
    for at in range(1, 9):
        out = moved(torch.zeros_like(x), at)
        same(calls(moved(x, at), moved(dw, at), moved(bias, at), out), want)
        around = out._base
        assert torch.isnan(around[:at]).all() and torch.isnan(around[at + T * E:]).all()


@pytest.mark.parametrize("E", [60, 252])
def test_rows_of_whole_pieces(E):
    """Rows of a multiple of four BF16 logits, which are eight bytes."""
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(41, E, device=DEV, generator=g).bfloat16()
    tail = x[1:]
    same(dg.moe_route(tail, 4), dg.moe_route(tail.clone(), 4))
    dw, ids = torch.ones(40, 4, device=DEV), dg.moe_route(tail, 4).ids
    assert torch.equal(dg.moe_route_bwd(dw, tail, ids), dg.moe_route_bwd(dw, tail.clone(), ids))


def test_refusals():
    """Rows of whole vectors have to lie at their alignment."""
    x, w = torch.zeros(70, device=DEV), torch.ones(70, device=DEV)
    for bad in (lambda: dg.residual_norm(x[1:65].view(4, 16), w_pre=w[:16]),
                lambda: dg.residual_norm(x[:64].view(4, 16), w_pre=w[1:17]),
                lambda: dg.moe_route(x[1:65].view(4, 16), 2), lambda: dg.moe_route(x.bfloat16()[2:66].view(4, 16), 2)):
        with pytest.raises(dg.DGError):
            bad()
