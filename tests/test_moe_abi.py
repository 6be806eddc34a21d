"""Argument checks of the mixture-of-experts operators (CPU only): every call
below fails validation or is empty work and returns before any HIP call; the
fake addresses are never dereferenced."""
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


SORT = dict(ids=P, it=0, T=100, k=2, G=8, align=128, M=2048, offs=P, counts=P, rs=P, sr=P, ws=P)


@pytest.mark.parametrize("kw,want", [
    (dict(it=2), INVALID), (dict(align=64), INVALID), (dict(align=0), INVALID), (dict(G=0), INVALID),
    (dict(T=-1), INVALID), (dict(T=BIG), INVALID), (dict(k=0), INVALID), (dict(M=-128), INVALID),
    (dict(M=1024), INVALID), (dict(M=2049), INVALID), (dict(ids=None), INVALID), (dict(ids=P + 2), INVALID),
    (dict(it=1, ids=P + 4), INVALID), (dict(offs=None), INVALID), (dict(counts=P + 1), INVALID),
    (dict(rs=None), INVALID), (dict(sr=None), INVALID), (dict(T=10000, M=1 << 20, ws=None), INVALID),
    (dict(G=1025, M=1 << 20), UNSUP), (dict(T=1 << 29, k=3, M=BIG - 128), UNSUP),
])
def test_sort_validation(kw, want):
    assert call(dg.dg_moe_sort, SORT, kw) == want


def test_rows_and_workspace():
    assert dg.dg_moe_rows(100, 2, 8, 128) == (200 + 127 * 8) // 128 * 128
    assert dg.dg_moe_rows(1, 2, 64, 128) == 256 and dg.dg_moe_rows(7, 3, 64, 1) == 21
    assert dg.dg_moe_rows(0, 2, 64, 128) == 0
    assert dg.dg_moe_rows(5, 0, 4, 1) == INVALID and dg.dg_moe_rows(5, 1, 4, 2) == INVALID
    assert dg.dg_moe_sort_workspace(100, 2, 8) == 0 and dg.dg_moe_sort_workspace(20000, 4, 8) > 0
    assert dg.dg_moe_sort_workspace(-1, 2, 8) == INVALID


PERMUTE = dict(X=P, dt=1, Y=P, sr=P, rs=P, T=10, k=2, M=512, H=256)
PERMUTE8 = dict(X=P, dt=1, Q=P, S=P, mode=1, sr=P, rs=P, T=10, k=2, M=512, H=256)
COMBINE = dict(Y=P, dt=1, w=P, sr=P, out=P, T=10, k=2, M=512, H=256)
COMBINE_BWD = dict(dO=P, Y=P, dt=1, w=P, sr=P, rs=P, dY=P, dw=P, T=10, k=2, M=512, H=256)


@pytest.mark.parametrize("fn,base", [(dg.dg_moe_permute, PERMUTE), (dg.dg_moe_permute_fp8, PERMUTE8),
                                     (dg.dg_moe_combine, COMBINE), (dg.dg_moe_combine_bwd, COMBINE_BWD)])
def test_token_operators_shared_validation(fn, base):
    for kw, want in [(dict(dt=2), INVALID), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(M=-1), INVALID),
                     (dict(H=-1), INVALID), (dict(H=BIG), INVALID), (dict(H=(1 << 22) + 16), UNSUP),
                     (dict(T=1 << 30, k=2), INVALID), (dict(T=1 << 29, k=3), UNSUP), (dict(sr=None), INVALID),
                     (dict(sr=P + 2), INVALID)]:
        assert call(fn, base, kw) == want, kw


@pytest.mark.parametrize("kw,want", [(dict(X=None), INVALID), (dict(Y=P + 8), INVALID), (dict(rs=None), INVALID),
                                     (dict(M=0), OK), (dict(H=0), OK)])
def test_permute_validation(kw, want):
    assert call(dg.dg_moe_permute, PERMUTE, kw) == want


@pytest.mark.parametrize("kw,want", [(dict(X=P + 4), INVALID), (dict(Q=None), INVALID), (dict(S=None), INVALID),
                                     (dict(S=P + 2), INVALID), (dict(mode=2), INVALID), (dict(H=200), UNSUP),
                                     (dict(rs=None), INVALID), (dict(M=0), OK), (dict(H=0), OK)])
def test_permute_fp8_validation(kw, want):
    assert call(dg.dg_moe_permute_fp8, PERMUTE8, kw) == want


@pytest.mark.parametrize("kw,want", [(dict(Y=None), INVALID), (dict(out=None), INVALID), (dict(w=P + 2), INVALID),
                                     (dict(out=P + 8), INVALID), (dict(T=0), OK), (dict(H=0), OK)])
def test_combine_validation(kw, want):
    assert call(dg.dg_moe_combine, COMBINE, kw) == want


@pytest.mark.parametrize("kw,want", [(dict(Y=None), INVALID), (dict(dO=None), INVALID), (dict(w=None), INVALID),
                                     (dict(dY=P + 8), INVALID), (dict(dw=None), INVALID), (dict(rs=None), INVALID),
                                     (dict(T=0, M=0), OK)])
def test_combine_bwd_validation(kw, want):
    assert call(dg.dg_moe_combine_bwd, COMBINE_BWD, kw) == want


SWIGLU = dict(H=P, dt=1, A=P, sA=P, Hq=P, sH=P, M=10, I=256)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=-1), INVALID), (dict(M=-1), INVALID), (dict(I=BIG), INVALID), (dict(Hq=None), INVALID),
    (dict(sH=None), INVALID), (dict(H=None), INVALID), (dict(A=P + 8), INVALID), (dict(sA=None), INVALID),
    (dict(Hq=P + 1), INVALID), (dict(I=24), UNSUP), (dict(I=(1 << 22) + 16), UNSUP), (dict(M=0), OK), (dict(I=0), OK),
])
def test_swiglu_validation(kw, want):
    assert call(dg.dg_swiglu_fp8, SWIGLU, kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), INVALID), (dict(M=BIG), INVALID), (dict(dA=None), INVALID), (dict(Hq=None), INVALID),
    (dict(sH=P + 2), INVALID), (dict(dH=P + 8), INVALID), (dict(I=8), UNSUP), (dict(M=0), OK), (dict(I=0), OK),
])
def test_swiglu_bwd_validation(kw, want):
    assert call(dg.dg_swiglu_fp8_bwd, dict(dA=P, dt=1, Hq=P, sH=P, dH=P, M=10, I=256), kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(out=2), INVALID), (dict(acc=2), INVALID), (dict(G=0), INVALID), (dict(M=-1), INVALID),
    (dict(N=BIG), INVALID), (dict(dY=None), INVALID), (dict(X=P + 8), INVALID), (dict(sX=None), INVALID),
    (dict(offs=None), INVALID), (dict(counts=P + 2), INVALID), (dict(dW=None), INVALID), (dict(N=20), UNSUP),
    (dict(K=24), UNSUP), (dict(N=0), OK), (dict(K=0), OK),
])
def test_wgrad_validation(kw, want):
    base = dict(dY=P, X=P, sX=P, offs=P, counts=P, G=4, M=512, N=256, K=256, dW=P, out=0, acc=0)
    assert call(dg.dg_grouped_wgrad_fp8, base, kw) == want


@pytest.mark.parametrize("kw", [dict(G=(1 << 23) + 1, N=8, K=16), dict(G=1 << 15, N=4096, K=4096)])
def test_wgrad_grid_limit(kw):
    base = dict(dY=P, X=P, sX=P, offs=P, counts=P, G=4, M=512, N=256, K=256, dW=P, out=0, acc=0)
    assert call(dg.dg_grouped_wgrad_fp8, base, kw) == UNSUP


def test_helpers_refuse_host_tensors_and_wrong_types():
    f, i = torch.zeros(4, 32), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        dg.moe_sort(f, 4)
    with pytest.raises(ValueError):
        dg.moe_sort(i, 4)                                       # not on the device
    with pytest.raises(ValueError):
        dg.moe_sort(i[0], 4)
    with pytest.raises(TypeError):
        dg.moe_permute(f.half(), i, i[:, 0])
    with pytest.raises(ValueError):
        dg.moe_combine(f[0], i)
    with pytest.raises(ValueError):
        dg.swiglu_fp8(f)
    with pytest.raises(ValueError):
        dg.scale_code("e8m0")
    with pytest.raises(ValueError):
        dg.grouped_wgrad_fp8(f[0], f, f, i[0])


def test_binding_refuses_what_is_not_a_tensor_or_a_number():
    f, i = torch.zeros(4, 32), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: dg.moe_sort([[0, 1]], 4), lambda: dg.moe_permute(f, None, i), lambda: dg.moe_combine(3, i),
                 lambda: dg.swiglu_fp8(None), lambda: dg.grouped_wgrad_fp8(f, f, f, "offsets")):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(TypeError):
        dg.binding().moe_sort(i)                                # too few arguments
    with pytest.raises(TypeError):
        dg.moe_sort(i.float(), 4)
    with pytest.raises(ValueError):
        dg.grouped_wgrad_fp8(f, f, f, i[0], out_dtype="f16")
