"""NaN and infinities of the normalised rows as E4M3 codes.  Needs a GPU.

A NaN has a NaN code, and the block's other codes and scale are those of its numbers,
whatever they are; a block with a value that FP32 does not hold has a NaN scale and NaN
codes.  Codes and scales are compared exactly."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import block as O
from oracle import moe as M
from test_gpu_norm import B, DEV, F, dev, n, problem

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def codes_of(p, codes):
    out = dg.residual_norm(dev(p["R"]), w_pre=dev(p["w_pre"]), codes=codes, values=False)
    torch.cuda.synchronize()
    return n(out.Q), n(out.S)


def is_nan(q):
    return (q & 0x7F) == 0x7F


@pytest.mark.parametrize("codes", ["pow2", "amax"])
@pytest.mark.parametrize("rt", [B, F])
def test_nan_has_a_nan_code_whatever_is_beside_it(codes, rt):
    """A NaN in each four columns of two million: some of the others are near a border
    between codes, where the four are computed again."""
    p = problem(4000, 512, rt, rt, block=False)
    bad = torch.arange(512) % 4 == torch.arange(512) // 4 % 4
    clean = p["w_pre"].clone()
    clean[bad] = 0
    p["w_pre"][bad] = NAN
    q, s = codes_of(p, codes)
    _, N, _ = O.residual_norm(n(p["R"]), w_pre=n(clean), eps=EPS)
    want, scales = M.quantise(N, codes == "pow2")
    bad = bad.numpy()
    assert np.array_equal(s, scales) and np.array_equal(q[:, ~bad], want[:, ~bad])
    assert is_nan(q[:, bad]).all()


@pytest.mark.parametrize("codes", ["pow2", "amax"])
def test_rows_of_nan(codes):
    """A NaN of the stream is its whole row's; a block without a number has the scale 1."""
    p = problem(9, 272, F, F, block=False)
    clean = codes_of(p, codes)
    p["R"][2, 5], p["R"][4, 1] = NAN, INF
    q, s = codes_of(p, codes)
    rows = [0, 1, 3, 5, 6, 7, 8]
    assert np.array_equal(q[rows], clean[0][rows]) and np.array_equal(s[rows], clean[1][rows])
    assert is_nan(q[2]).all() and (s[2] == 1).all()
    assert is_nan(q[4, 1]) and not (q[4, 2:] & 0x7F).any() and (s[4] == 1).all()     # (the others over infinity)


@pytest.mark.parametrize("codes", ["pow2", "amax"])
@pytest.mark.parametrize("weight", [INF, -INF, 3e38])
def test_blocks_past_fp32(codes, weight):
    """Weights that bring a column past FP32's largest number: its block is NaN in those rows."""
    p = problem(300, 400, F, F, block=False)
    p["w_pre"][200] = weight
    p["w_pre"][7] = 1e38                                      # in range, with values up to about 4
    p["R"][:, 7].clamp_(-2, 2)
    x = n(p["R"])
    unit = x * O.rstd(x, EPS)
    past = np.abs(unit[:, 200]) * abs(weight) > float(torch.finfo(F).max)
    assert past.any() and np.abs(unit[:, 7]).max() < 3
    q, s = codes_of(p, codes)
    w = n(p["w_pre"]).copy()
    if np.isinf(weight):
        assert past.all()
        w[200] = 0
    want, scales = M.quantise(unit * w, codes == "pow2")
    block = np.arange(400) // 128 == 1
    ok = np.ones(s.shape, bool)
    ok[past, 1] = False
    assert np.array_equal(s[ok], scales[ok]) and np.isnan(s[~ok]).all()
    assert np.array_equal(q[:, ~block], want[:, ~block]) and np.array_equal(q[~past], want[~past])
    assert is_nan(q[past][:, block]).all()
