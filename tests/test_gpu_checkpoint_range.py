"""The gated activation's gradient over the whole range of what a checkpoint can
hold: gates far out on both sides, NaN, and products that leave FP32's range on
the way to a result inside it.  Checkpoints are made directly, as codes and
scales.  Needs a GPU.

Tolerance.  The factors' relative errors are as in test_gpu_checkpoint.py: 2^-20
of the magnitudes of the terms, and half a step (2^-8) for a BF16 result.  The
only absolute term is FP32's smallest step, 2^-149, for an FP32 result and the
smallest normal number, 2^-126, for a BF16 one."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import moe as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN_CODE = 0x7F


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def checkpoint(g, u):
    """(codes, scales) of [M][I] gates and factors, exactly as the oracle quantises."""
    (qg, sg), (qu, su) = O.quantise(g, True), O.quantise(u, True)
    return np.concatenate([qg, qu], 1), np.stack([sg, su], 1)


def run(da, Hq, sH, dtype):
    """(dg, du) of the kernel and dA as it saw it, in float64."""
    d = torch.from_numpy(np.ascontiguousarray(da)).to(DTYPE[dtype]).to(DEV)
    dH = dg.swiglu_fp8_bwd(d, torch.from_numpy(Hq).to(DEV), torch.from_numpy(np.ascontiguousarray(sH)).to(DEV))
    torch.cuda.synchronize()
    I = da.shape[1]
    got = dH.double().cpu().numpy()
    return got[:, :I], got[:, I:], d.double().cpu().numpy()


def decoded(Hq, sH, I):
    return (O.dequantise(Hq[:, i * I:(i + 1) * I], np.ascontiguousarray(sH[:, i])) for i in (0, 1))


def check(da, Hq, sH, dtype):
    I = da.shape[1]
    got_g, got_u, d = run(da, Hq, sH, dtype)
    g, u = decoded(Hq, sH, I)
    with np.errstate(over="ignore"):
        want_g, want_u, mass = O.swiglu_bwd(d, g, u)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    least = 2.0 ** -126 if dtype == "bf16" else 2.0 ** -149
    top = float(torch.finfo(DTYPE[dtype]).max)
    for name, got, want, m in (("dg", got_g, want_g, mass), ("du", got_u, want_u, np.abs(want_u))):
        bound = half * np.abs(want) + 2.0 ** -20 * m + least
        ok = np.abs(got - want) <= bound
        ok |= (np.abs(want) + bound > top) & np.isinf(got) & (np.sign(got) == np.sign(want))
        bad = np.argwhere(~ok)
        assert not len(bad), [(name, i.tolist(), float(g[tuple(i)]), float(u[tuple(i)]), float(got[tuple(i)]),
                               float(want[tuple(i)])) for i in bad[:4]]


FAR = (-3.3e38, -1e36, -1e33, -1e30, -1e20, -1e6, -1000.0, -300.0, -150.0, -120.0, -104.0, -100.0, -96.0, -90.0,
       -88.0, -87.0, -81.0, -80.0, -72.0, -64.0, -60.0, -57.0, -56.0, -52.0, -40.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 40, 2.0 ** 90])
def test_far_negative_gates(dtype, size):
    """The gradient goes to 0 with the gate, as e^g does: 0 at the far end, and
    right relative to itself where a large u brings it back into range."""
    log(f"far negative gates {dtype} size={size:g}")
    rng = np.random.default_rng(1)
    g = np.repeat(np.array(FAR)[:, None], 144, 1)              # a whole block and a partial one
    u = rng.standard_normal(g.shape) * size
    check(rng.standard_normal(g.shape), *checkpoint(g, u), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_gates_beside_ordinary_ones(dtype):
    """Within one block, and with positive gates as far out."""
    rng = np.random.default_rng(2)
    g = rng.standard_normal((64, 272)) * np.exp2(rng.uniform(-2, 9, (64, 1)))
    g[::5, 3] = 448 * 2.0 ** 119
    g[1::5, 7] = -3.35e38                                      # its code rounds up to 2^128
    u = rng.standard_normal(g.shape)
    check(rng.standard_normal(g.shape), *checkpoint(g, u), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["gate code", "factor code", "gate scale", "factor scale"])
@pytest.mark.parametrize("scale", [2.0 ** -9, 1.0])
def test_nan_reaches_the_gradient(dtype, where, scale):
    """A NaN in the checkpoint is a NaN in what depends on it, and nowhere else."""
    I = 256
    rng = np.random.default_rng(3)
    Hq, sH = checkpoint(rng.standard_normal((3, I)) * 300 * scale, rng.standard_normal((3, I)) * 300 * scale)
    da = rng.standard_normal((3, I))
    clean = run(da, Hq, sH, dtype)
    if where == "gate code":
        Hq[1, 5] = NAN_CODE
        hit_g, hit_u = (slice(5, 6),) * 2
    elif where == "factor code":
        Hq[1, I + 5] = NAN_CODE | 0x80
        hit_g, hit_u = slice(5, 6), slice(0, 0)
    elif where == "gate scale":
        sH[1, 0, 1] = np.nan
        hit_g, hit_u = (slice(128, 256),) * 2
    else:
        sH[1, 1, 1] = np.nan
        hit_g, hit_u = slice(128, 256), slice(0, 0)
    got = run(da, Hq, sH, dtype)
    for c, v, hit in ((clean[0], got[0], hit_g), (clean[1], got[1], hit_u)):
        want = np.zeros(v.shape, bool)
        want[1, hit] = True
        assert np.array_equal(np.isnan(v), want), where
        assert np.array_equal(v[~want], c[~want]), where


# gate, factor and incoming gradient: the result is in range, a product on the way is not
PRODUCTS = [(-56.0, 1e25, 1e20), (-60.0, 1e25, 1e20), (-40.0, 1e30, 1e15), (1.0, 1e-30, 1e30), (1.0, 1e30, 1e-30),
            (-52.0, 1e-30, 1e38), (3.0, 3.0e38, 1e-3), (44.0, 3.0e38, 1e-20), (1e-38, 1.0, 1e38), (1e-35, 1e-5, 1e30),
            (1e-30, 1e-30, 1e30), (3e38, 2.0, 1e-3), (3e38, 1e-38, 1e-3), (-80.0, 1e38, 1e30), (20.0, 1e-38, 1e38),
            (-56.0, 2.0 ** -40, 1e38), (-56.0, 2.0 ** 100, 1.0), (2.0 ** -50, 1.0, 1e38)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products_that_leave_the_range_on_the_way(dtype):
    rng = np.random.default_rng(4)
    rows = np.array(PRODUCTS)
    wobble = lambda: 1 + rng.uniform(0, 0.1, (len(rows), 144))
    g, u, da = (rows[:, i:i + 1] * wobble() for i in range(3))
    top = 3.38e38                                              # dA itself is finite
    check(np.clip(da, -top, top), *checkpoint(np.clip(g, -top, top), np.clip(u, -top, top)), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_random_exponents(dtype):
    """Gates, factors and gradients of any size against each other."""
    rng = np.random.default_rng(5)
    M, I = 256, 144
    size = lambda lo, hi: np.exp2(rng.uniform(lo, hi, (M, 1)))
    g = rng.uniform(-1, 1, (M, I)) * size(-120, 127)
    g[::2] = rng.uniform(-1, 1, (M // 2, I)) * size(-8, 8)[::2]
    u = rng.uniform(-1, 1, (M, I)) * size(-126, 127)
    check(rng.uniform(-1, 1, (M, I)) * size(-100, 126), *checkpoint(g, u), dtype)
