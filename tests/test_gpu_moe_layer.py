"""The operators of a mixture-of-experts layer put together (examples/moe_layer.py):
every stage of a training step against the float64 oracle on the stage's own
inputs, the step under graph capture, and decode.  Needs a GPU."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_gemm_block_amd import dg
from oracle import moe as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def setup(example, E=5, H=256, I=384, T=150, k=2, drop=0.1, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    layer = example.MoELayer(E, H, I, generator=g)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    ids, w = example.route(x, torch.randn(H, E, device=DEV, generator=g), k)
    ids = torch.where(torch.rand(T, k, device=DEV, generator=g) < drop, -1, ids)
    dout = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    return layer, x, ids, w, dout


def n(t):
    return (t.double() if t.is_floating_point() else t).cpu().numpy()


def check_product(C, A, sA, W, Ws, plan):
    """A grouped product against the oracle, expert by expert; padding is zero."""
    C, A, sA, W, Ws = n(C), n(A), sA.cpu().numpy(), n(W), Ws.cpu().numpy()
    offs, counts = n(plan.group_offsets), n(plan.group_counts)
    real = np.zeros(C.shape[0], bool)
    for e in range(len(counts)):
        r = slice(offs[e], offs[e] + counts[e])
        real[r] = True
        if counts[e] == 0:
            continue
        a = O.dequantise(A[r], sA[r])
        w = oracle.decode_table()[W[e]] * np.kron(Ws[e].astype(np.float64), np.ones((128, 128)))
        want, mass = a @ w.T, np.abs(a) @ np.abs(w).T
        assert np.all(np.abs(C[r] - want) <= oracle.tolerance(want, mass, "bf16"))
    assert not C[~real].any()


def test_training_step_stage_by_stage(example):
    layer, x, ids, w, dout = setup(example)
    out, saved = layer.forward(x, ids, w)
    plan, _, xq, sx, a, sa, hq, sh, y = saved
    h = dg.grouped_gemm_fp8(xq, sx, layer.q13.q, layer.q13.s, plan.group_offsets, group_counts=plan.group_counts)
    torch.cuda.synchronize()
    ref = O.sort(n(ids), layer.experts, 128, len(plan.row_slot))
    for got, want in zip(plan, ref):
        assert np.array_equal(n(got), want)
    q, s = O.quantise(n(x), True)
    assert np.array_equal(n(xq), O.permute(q, ref[2], 2)) and np.array_equal(sx.cpu().numpy(), O.permute(s, ref[2], 2, fill=1))
    check_product(h, xq, sx, layer.q13.q, layer.q13.s, plan)
    I = layer.inner
    act, act_s = O.quantise(O.swiglu(n(h)[:, :I], n(h)[:, I:]), True)
    assert np.array_equal(n(a) & 0x7F, act & 0x7F) and np.array_equal(sa.cpu().numpy(), act_s)
    check_product(y, a, sa, layer.q2.q, layer.q2.s, plan)
    want, mass = O.combine(n(y), ref[3], n(w))
    assert np.all(np.abs(n(out) - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -24 * mass)

    dx, dweights, dw13, dw2 = layer.backward(dout, saved)
    dy, dweights2 = dg.moe_combine_bwd(dout, y, plan.slot_row, plan.row_slot, w)
    da = dg.grouped_gemm_fp8(*dg.quantize_fp8_blockscaled(dy, 1), layer.q2.qt, layer.q2.st, plan.group_offsets,
                             group_counts=plan.group_counts)
    dh = dg.swiglu_fp8_bwd(da, hq, sh)
    torch.cuda.synchronize()
    assert torch.equal(dweights, dweights2)
    dq, ds = dg.quantize_fp8_blockscaled(dy, 1)
    check_product(da, dq, ds, layer.q2.qt, layer.q2.st, plan)
    for got, d, codes, scales in ((dw2, dy, a, sa), (dw13, dh, xq, sx)):
        want, mass = O.wgrad(n(d), O.dequantise(n(codes), scales.cpu().numpy()), ref[0], ref[1])
        rows = ref[1].reshape(-1, 1, 1) + 1
        # each FP32 sum is off by at most a step of the magnitudes
        assert np.all(np.abs(n(got) - want) <= rows * 2.0 ** -23 * mass + 2.0 ** -24 * np.abs(want))
    assert dx.shape == x.shape and bool(torch.isfinite(dx.float()).all())


def test_gradients_follow_the_loss(example):
    """A step along the weight gradients lowers the loss by what they say, within
    the 8-bit operands' errors (each of the four products' operands is off by at
    most 2^-4 of itself)."""
    layer, x, ids, w, dout = setup(example, T=500, drop=0.0)
    loss = lambda: float((layer.forward(x, ids, w)[0].double() * dout.double()).sum())
    _, saved = layer.forward(x, ids, w)
    grad = layer.backward(dout, saved)[3]
    # along W2 the loss is linear but for the weights' own rounding: a step as
    # large as the weights keeps that small next to it
    base = layer.w2.clone()
    step = grad / grad.square().mean().sqrt() * base.square().mean().sqrt()
    values = []
    for sign in (1, -1):
        layer.w2.copy_(base + sign * step)
        layer.refresh()
        values.append(loss())
    want = 2 * float((grad.double() * step.double()).sum())
    log(f"difference {values[0] - values[1]:.6g}, gradient {want:.6g}")
    assert abs(values[0] - values[1] - want) <= 2.0 ** -4 * want


def test_step_under_graph_capture(example):
    layer, x, ids, w, dout = setup(example, T=700, k=2)

    def step():
        out, saved = layer.forward(x, ids, w)
        return (out, *layer.backward(dout, saved))

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                        # the stream's workspace exists before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        other = step()                                # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b, c) in enumerate(zip(got, want, other)):
            assert torch.equal(a, b) and torch.equal(c, b), f"replay {rep}: output {i}"


def test_large_sort_under_graph_capture():
    """The sort of two launches with its workspace."""
    ids = torch.randint(-1, 64, (5000, 4), device=DEV)
    x = torch.randn(5000, 144, device=DEV)

    def step():
        plan = dg.moe_sort(ids, 64)
        return (*plan, *dg.moe_permute_fp8(x, plan.slot_row, plan.row_slot))

    want = [t.clone() for t in step()]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        got = step()
    for rep in range(4):
        for t in got:
            t.zero_()
        other = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, other):
            assert torch.equal(a, b) and torch.equal(c, b), rep


@pytest.mark.parametrize("T", [1, 3, 64])
def test_decode(example, T):
    """Packed segments give each token what the padded ones do: the same codes,
    and products that differ by their roundings only."""
    layer, x, ids, w, _ = setup(example, T=T, drop=0.0)
    got, want = layer.decode(x, ids, w), layer.forward(x, ids, w)[0]
    torch.cuda.synchronize()
    # h and y are rounded to BF16 (2^-8) after sums in another order: a code of the
    # activation may move by one step, 2^-3 of it, where h moves by a rounding step
    err = float((got.double() - want.double()).norm() / want.double().norm())
    log(f"decode T={T}: {err:.2e}")
    assert err <= 2.0 ** -6
