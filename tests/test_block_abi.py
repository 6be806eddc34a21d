"""Argument checks of the router, the norms around a block and clipping (CPU only):
every call below fails validation or is empty work and returns before any HIP call; the
fake addresses are never dereferenced."""
import ctypes
import math

import pytest
import torch

from moe_grouped_gemm_block_amd import dg

OK, INVALID, UNSUP = dg.DG_OK, dg.DG_ERR_INVALID_ARG, dg.DG_ERR_UNSUPPORTED
P = 1 << 20
BIG = 1 << 31


def call(fn, defaults, kw):
    d = dict(defaults)
    d.update(kw)
    return fn(*d.values(), None)


ROUTE = dict(x=P, dt=0, bias=None, mask=None, T=10, E=64, k=2, score=0, renorm=1, scale=1.0, ids=P, w=P, counts=P,
             sums=P, routed=P, loss=P, ws=P)
ROUTE_BWD = dict(dw=P, x=P, dt=0, ids=P, counts=P, routed=P, dloss=P, T=10, E=64, k=2, score=0, renorm=1, scale=1.0,
                 dx=P)
SHARED = [(dict(dt=2), INVALID), (dict(T=-1), INVALID), (dict(T=BIG), INVALID), (dict(E=0), INVALID),
          (dict(k=0), INVALID), (dict(E=4, k=5), INVALID), (dict(E=1025), UNSUP), (dict(k=65, E=100), UNSUP),
          (dict(T=1 << 30, k=2), INVALID), (dict(T=1 << 29, k=3), UNSUP), (dict(score=2), INVALID),
          (dict(renorm=2), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
          (dict(x=None), INVALID), (dict(x=P + 8), INVALID), (dict(ids=None), INVALID), (dict(ids=P + 2), INVALID),
          (dict(counts=None), INVALID), (dict(routed=None), INVALID), (dict(counts=P + 1), INVALID)]


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(w=None), INVALID), (dict(bias=P + 2), INVALID), (dict(sums=None), INVALID), (dict(loss=None), INVALID),
    (dict(loss=P + 2), INVALID), (dict(T=1000, ws=None), INVALID), (dict(T=1000, ws=P + 4), INVALID)])
def test_route_validation(kw, want):
    assert call(dg.dg_moe_route, ROUTE, kw) == want


@pytest.mark.parametrize("kw,want", SHARED + [(dict(dw=None), INVALID), (dict(dx=None), INVALID),
                                              (dict(dx=P + 4), INVALID), (dict(dloss=None), INVALID)])
def test_route_bwd_validation(kw, want):
    assert call(dg.dg_moe_route_bwd, ROUTE_BWD, kw) == want


def test_route_empty_work_and_workspace():
    none = dict(counts=None, sums=None, routed=None, loss=None, ws=None)
    assert call(dg.dg_moe_route, ROUTE, dict(none, T=0, x=None, ids=None, w=None)) == OK
    assert call(dg.dg_moe_route_bwd, ROUTE_BWD, dict(T=0, x=None, ids=None, dw=None, dx=None)) == OK
    assert dg.dg_moe_route_workspace(0, 64, 2) == dg.dg_moe_route_workspace(20, 64, 2) == 0
    assert dg.dg_moe_route_workspace(1000, 64, 2) > 0 and dg.dg_moe_route_workspace(1 << 29, 1024, 2) > 0
    for T, E, k, want in [(-1, 4, 1, INVALID), (5, 0, 1, INVALID), (5, 4, 5, INVALID), (5, 1025, 1, UNSUP),
                          (5, 100, 65, UNSUP)]:
        assert dg.dg_moe_route_workspace(T, E, k) == want


NORM = dict(R=P, rt=1, Y=2 * P, dt=1, w_post=P, gate=P, kind=1, alpha=1.0, w_pre=P, eps=1e-6, Ro=3 * P, N=4 * P, Q=P,
            S=P, mode=1, T=10, H=256)
NORM_BWD = dict(dR=5 * P, dN=6 * P, R=P, rt=1, Y=2 * P, dt=1, w_post=P, gate=P, kind=1, alpha=1.0, w_pre=P, eps=1e-6,
                dRo=3 * P, dY=4 * P, dwp=P, dg=P, dwr=P, T=10, H=256, ws=P)
NORMS = [(dict(rt=2), INVALID), (dict(dt=-1), INVALID), (dict(kind=3), INVALID), (dict(kind=0), INVALID),
         (dict(gate=None), INVALID), (dict(alpha=math.nan), INVALID), (dict(eps=0.0), INVALID),
         (dict(eps=-1.0), INVALID), (dict(eps=math.inf), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
         (dict(H=BIG), INVALID), (dict(H=(1 << 22) + 16), UNSUP), (dict(R=None), INVALID), (dict(R=P + 8), INVALID),
         (dict(Y=None), INVALID), (dict(Y=2 * P + 8), INVALID), (dict(w_post=P + 4), INVALID),
         (dict(gate=P + 4), INVALID), (dict(w_pre=P + 8), INVALID)]


@pytest.mark.parametrize("kw,want", NORMS + [
    (dict(mode=2), INVALID), (dict(Ro=None), INVALID), (dict(Ro=P), INVALID), (dict(Ro=2 * P), INVALID),
    (dict(N=P), INVALID), (dict(N=4 * P + 8), INVALID), (dict(Q=None), INVALID), (dict(S=None), INVALID),
    (dict(Q=P + 8), INVALID), (dict(w_pre=None), INVALID), (dict(N=None, Q=None, S=None), INVALID), (dict(H=250), UNSUP),
    (dict(Y=None, w_post=None, gate=None, kind=0), INVALID),
    (dict(Y=None, w_post=None, gate=None, kind=0, Ro=None, w_pre=None, N=None, Q=None, S=None), INVALID)])
def test_norm_validation(kw, want):
    assert call(dg.dg_residual_norm, NORM, kw) == want


@pytest.mark.parametrize("kw,want", NORMS + [
    (dict(dRo=None), INVALID), (dict(dRo=P), INVALID), (dict(dRo=5 * P), INVALID), (dict(dRo=4 * P), INVALID),
    (dict(dY=None), INVALID), (dict(dY=2 * P), INVALID), (dict(dY=6 * P), INVALID), (dict(dN=None), INVALID),
    (dict(dR=5 * P + 4), INVALID), (dict(dwp=None), INVALID), (dict(dg=None), INVALID), (dict(dwr=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws=P + 4), INVALID), (dict(w_pre=None, dwr=None, R=None), INVALID),
    (dict(w_pre=None, dwr=None, dN=None, dR=None), INVALID), (dict(w_post=None), INVALID)])
def test_norm_bwd_validation(kw, want):
    assert call(dg.dg_residual_norm_bwd, NORM_BWD, kw) == want


def test_norm_empty_work_and_workspace():
    assert call(dg.dg_residual_norm, NORM, dict(T=0, R=None, Ro=None, N=None, Q=None, S=None)) == OK
    assert call(dg.dg_residual_norm_bwd, NORM_BWD, dict(T=0, w_pre=None, dwr=None, w_post=None, dwp=None, gate=None,
                                                        dg=None, kind=0)) == OK
    assert dg.dg_residual_norm_bwd_workspace(0, 256, 2) == 0
    assert dg.dg_residual_norm_bwd_workspace(100, 256, 2) == 2 * dg.dg_residual_norm_bwd_workspace(100, 256, 1) > 0
    assert dg.dg_residual_norm_bwd_workspace(1 << 20, 1 << 22, 2) <= 64 << 20
    for T, H, n, want in [(-1, 8, 1, INVALID), (1, 0, 1, INVALID), (1, 8, 3, INVALID), (1, (1 << 22) + 1, 1, UNSUP)]:
        assert dg.dg_residual_norm_bwd_workspace(T, H, n) == want


def arrays(tensors):
    """(addresses, sizes, dtypes, count) of (address, size, dtype)."""
    n = len(tensors)
    return ((ctypes.c_void_p * n)(*(t[0] for t in tensors)), (ctypes.c_int64 * n)(*(t[1] for t in tensors)),
            (ctypes.c_int * n)(*(t[2] for t in tensors)), n)


def norm_of(tensors, norm=P, ws=P):
    g, s, d, n = arrays(tensors)
    return dg.dg_grad_norm(g, s, d, n, norm, ws, None)


def clip_of(tensors, outs, norm=P, max_norm=1.0):
    g, s, d, n = arrays(tensors)
    o, _, od, _ = arrays([(a, 0, t) for a, t in outs])
    return dg.dg_clip_grads(g, s, d, n, norm, max_norm, o, od, None)


def test_grad_norm_validation():
    one = [(P, 10, 0)]
    assert norm_of(one, norm=None) == INVALID and norm_of(one, norm=P + 2) == INVALID
    large = [(P, 100000, 0)]
    assert norm_of(large, ws=None) == INVALID and norm_of(large, ws=P + 4) == INVALID
    for t in [(None, 10, 0), (P + 2, 10, 0), (P + 1, 10, 1), (P, -1, 0), (P, 10, 2), (P, 1 << 46, 0)]:
        assert norm_of([t]) == INVALID, t
    assert dg.dg_grad_norm(None, None, None, 1, P, P, None) == INVALID
    assert dg.dg_grad_norm(None, None, None, -1, P, P, None) == INVALID
    assert norm_of([(P, 1 << 45, 0)]) == UNSUP
    _, s, d, n = arrays([(P, 0, 0), (P, 1, 1), (P, 1 << 20, 0)])
    assert dg.dg_grad_norm_workspace(s, d, n) >= 16 and dg.dg_grad_norm_workspace(s, d, 1) == 0
    assert dg.dg_grad_norm_workspace(s, d, -1) == INVALID


def test_clip_validation():
    one = [(P, 10, 0)]
    assert clip_of(one, [(P, 0)], norm=None) == INVALID
    for m in (0.0, -1.0, math.inf, math.nan):
        assert clip_of(one, [(P, 0)], max_norm=m) == INVALID
    assert clip_of(one, [(P, 1)]) == INVALID                  # in place, of another type
    assert clip_of(one, [(None, 0)]) == INVALID and clip_of(one, [(2 * P + 2, 0)]) == INVALID
    assert clip_of(one, [(2 * P, 2)]) == INVALID
    two = [(P, 10, 0), (2 * P, 10, 0)]
    for outs in ([(3 * P, 0), (3 * P, 0)], [(3 * P, 0), (3 * P + 36, 0)], [(2 * P, 0), (P, 0)],
                 [(P, 0), (P + 20, 0)], [(P + 20, 0), (3 * P, 0)], [(2 * P + 36, 0), (3 * P, 0)]):
        assert clip_of(two, outs) == INVALID, outs
    assert clip_of([(P, 10, 0), (P, 10, 0)], [(P, 0), (P, 0)]) == INVALID     # the same tensor twice, in place
    assert clip_of([(P, 0, 0)], [(None, 0)]) == OK and clip_of([], []) == OK   # nothing to do


@pytest.mark.parametrize("norm", [P, P + 36, P + 4 * 9999])
def test_clip_refuses_to_write_over_its_norm(norm):
    for n, g in ((10, 2 * P), (10, P), (10000, P)):
        if P <= norm < P + 4 * n:
            assert clip_of([(g, n, 0)], [(P, 0)], norm=norm) == INVALID
            assert clip_of([(2 * P, 5, 0), (g + (g == 2 * P) * P, n, 0)], [(4 * P, 0), (P, 0)], norm=norm) == INVALID


# ---------------------------------------------------------------- the torch side, on the CPU

def test_binding_refuses_what_is_no_device_tensor():
    x = torch.zeros(4, 8)
    for fn in (lambda: dg.moe_route(x, 2), lambda: dg.residual_norm(x, w_pre=torch.ones(8)),
               lambda: dg.grad_norm([x]), lambda: dg.clip_grads([x], torch.ones(()), 1.0),
               lambda: dg.residual_norm_bwd(x, x, x, w_pre=torch.ones(8)),
               lambda: dg.moe_route_bwd(x, x, torch.zeros(4, 8, dtype=torch.int32))):
        with pytest.raises(ValueError, match="contiguous device tensor"):
            fn()


def test_binding_refuses_other_types_and_names():
    x = torch.zeros(4, 8)
    for fn in (lambda: dg.moe_route(x.half(), 2), lambda: dg.moe_route("x", 2), lambda: dg.grad_norm(x),
               lambda: dg.grad_norm([x.half()]), lambda: dg.clip_grads({0: x}, x, 1.0),
               lambda: dg.residual_norm(x.double())):
        with pytest.raises(TypeError):
            fn()
    for fn in (lambda: dg.moe_route(x, 2, score="tanh"), lambda: dg.residual_norm(x, codes="int8"),
               lambda: dg.residual_norm(x, dtype="f16"), lambda: dg.moe_route(x[0], 2), lambda: dg.grad_norm([])):
        with pytest.raises(ValueError):
            fn()
