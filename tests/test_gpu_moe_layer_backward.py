"""The backward pass of examples/moe_layer.py: each of its stages against the
float64 oracle on the stage's own inputs, and all of its gradients against
differences of the loss.  Needs a GPU.

Tolerances.  A BF16 result is off by half a step, 2^-8; products and sums in FP32
by 2^-24 of the magnitudes for each operation (a sum of n terms: n of them,
however ordered); the gated activation's factors by 2^-20 (test_gpu_checkpoint.py).
The stages are called again here with the layer's own tensors; results repeat
bit for bit, so what the layer returns has to be equal to them."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import moe as O
from test_gpu_moe_layer import check_product, example, n, setup  # noqa: F401  (example: a fixture)

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def check(got, want, mass, fp32_steps):
    bound = HALF * np.abs(want) + fp32_steps * 2.0 ** -24 * mass + 2.0 ** -126
    err = np.abs(n(got) - want)
    assert np.all(err <= bound), float((err / bound).max())


def check_quantised(q, s, x):
    codes, scales = O.quantise(n(x), False)
    assert np.array_equal(n(q), codes) and np.array_equal(s.cpu().numpy(), scales)


def test_backward_stage_by_stage(example):
    layer, x, ids, w, dout = setup(example, seed=3)
    _, saved = layer.forward(x, ids, w)
    plan, _, xq, sx, a, sa, hq, sh, y = saved
    offs, counts, slot_row = (n(t) for t in (plan.group_offsets, plan.group_counts, plan.slot_row))
    dx, dweights, dw13, dw2 = layer.backward(dout, saved)

    dy, dw = dg.moe_combine_bwd(dout, y, plan.slot_row, plan.row_slot, w)
    qy, sy = dg.quantize_fp8_blockscaled(dy, 1)
    da = dg.grouped_gemm_fp8(qy, sy, layer.q2.qt, layer.q2.st, plan.group_offsets, group_counts=plan.group_counts)
    dh = dg.swiglu_fp8_bwd(da, hq, sh)
    qh, sqh = dg.quantize_fp8_blockscaled(dh, 1)
    drows = dg.grouped_gemm_fp8(qh, sqh, layer.q13.qt, layer.q13.st, plan.group_offsets, group_counts=plan.group_counts)
    torch.cuda.synchronize()

    want_y, want_w, mass_w = O.combine_bwd(n(dout), n(y), slot_row, n(w))
    check(dy, want_y, np.abs(want_y), 1)
    assert np.all(np.abs(n(dw) - want_w) <= layer.hidden * 2.0 ** -24 * mass_w + 2.0 ** -24 * np.abs(want_w))
    assert torch.equal(dw, dweights)
    check_quantised(qy, sy, dy)
    check_product(da, qy, sy, layer.q2.qt, layer.q2.st, plan)
    I = layer.inner
    g, u = (O.dequantise(n(hq)[:, i * I:(i + 1) * I], sh[:, i].cpu().numpy()) for i in (0, 1))
    want_g, want_u, mass_g = O.swiglu_bwd(n(da), g, u)
    check(dh[:, :I], want_g, mass_g, 16)
    check(dh[:, I:], want_u, np.abs(want_u), 16)
    check_quantised(qh, sqh, dh)
    check_product(drows, qh, sqh, layer.q13.qt, layer.q13.st, plan)
    want_x, mass_x = O.combine(n(drows), slot_row, None)
    check(dx, want_x, mass_x, ids.shape[1])
    for got, d, codes, scales in ((dw2, dy, a, sa), (dw13, dh, xq, sx)):
        want, mass = O.wgrad(n(d), O.dequantise(n(codes), scales.cpu().numpy()), offs, counts)
        rows = counts.reshape(-1, 1, 1) + 1
        assert np.all(np.abs(n(got) - want) <= rows * 2.0 ** -23 * mass + 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("what", ["x", "weights", "gate rows of w13", "factor rows of w13", "w2"])
def test_every_gradient_follows_the_loss(example, what):
    """A step along each gradient changes the loss by what the gradient says.
    Steps of an eighth of the values' size: small next to the activation's
    curvature (its third order: 2^-6 / 6 of the difference), large next to the
    rounding of single 8-bit operands, which averages out over 10^5 of them; the
    gradient's own operands are off by at most 2^-4 of themselves each."""
    layer, x, ids, w, dout = setup(example, T=500, drop=0.0)
    loss = lambda x, w: float((layer.forward(x, ids, w)[0].double() * dout.double()).sum())
    _, saved = layer.forward(x, ids, w)
    dx, dweights, dw13, dw2 = layer.backward(dout, saved)
    I = layer.inner
    rows = slice(0, I) if what.startswith("gate") else slice(I, 2 * I)
    value, grad = {"x": (x, dx), "weights": (w, dweights), "w2": (layer.w2, dw2)}.get(
        what, (layer.w13[:, rows], dw13[:, rows]))
    grad = grad.float()
    base = value.float().clone()
    step = grad / grad.square().mean().sqrt() * base.square().mean().sqrt() / 8
    values, steps = [], []
    for sign in (1, -1):
        value.copy_(base + sign * step)                        # x: rounded to BF16, and stepped by what is left
        steps.append(value.double() - base.double())
        layer.refresh()
        values.append(loss(x, w))
    want = float((grad.double() * (steps[0] - steps[1])).sum())
    log(f"{what}: difference {values[0] - values[1]:.6g}, gradient {want:.6g}")
    assert want > 0 and abs(values[0] - values[1] - want) <= 2.0 ** -4 * want
