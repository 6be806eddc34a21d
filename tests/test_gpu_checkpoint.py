"""The gated activation with its 8-bit checkpoint, its gradient, and the weight
gradient from 8-bit activations, against the float64 oracle.  Needs a GPU.

Tolerances.  Codes and scales are decisions about real numbers: they have to be
equal.  Gradients: e^-g is within 2^-22, the reciprocal within 2^-23, every
other operation within 2^-24, so each factor of dg and du is within 2^-20 of the
magnitude of its terms; a BF16 result adds half a step, 2^-8.  Weight gradients:
products of BF16 values are exact in FP32, each of the n sums is off by at most a
step, 2^-23 of the magnitudes, however the matrix core orders and truncates."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import moe as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def gate_values(M, I, rng):
    """(g, u): ordinary rows, padding, gates far out on both sides, tiny and large
    factors, and products close to a border between two codes."""
    g = rng.standard_normal((M, I)) * 3
    u = rng.standard_normal((M, I)) * 2
    for m in range(M):
        kind = m % 8
        if kind == 1:
            g[m] = u[m] = 0
        elif kind == 2:
            g[m] = rng.uniform(-120, 120, I)
        elif kind == 3:
            g[m] = rng.uniform(-130, -70, I)                     # every product tiny
            u[m] *= np.exp2(rng.uniform(0, 60))
        elif kind == 4:
            u[m] *= np.exp2(rng.uniform(-100, 100))
        elif kind == 5:
            g[m] *= np.exp2(rng.uniform(-60, 0))
        elif kind == 6:
            g[m] = 40                                            # u g / (1 + 4e-18): at the border itself
            u[m] = rng.choice([17, 19, 21, 23, 448, 0.0625], I) / 40
    return g, u


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,I", [(1, 16), (17, 128), (64, 176), (40, 1424), (130, 2048)])
def test_swiglu(M, I, dtype):
    log(f"swiglu M={M} I={I} {dtype}")
    g, u = gate_values(M, I, np.random.default_rng(M + I))
    h = torch.from_numpy(np.concatenate([g, u], 1)).to(DTYPE[dtype]).to(DEV)
    A, sA, Hq, sH = dg.swiglu_fp8(h)
    A2, sA2, none, none2 = dg.swiglu_fp8(h, checkpoint=False)
    torch.cuda.synchronize()
    hd = h.double().cpu().numpy()
    with np.errstate(over="ignore"):
        a = O.swiglu(hd[:, :I], hd[:, I:])
    codes, scales = O.quantise(a, True)
    assert np.array_equal(sA.cpu().numpy(), scales)
    diff = np.argwhere((A.cpu().numpy() & 0x7F) != (codes & 0x7F))
    assert diff.shape[0] == 0, [(i.tolist(), hd[i[0], i[1]], hd[i[0], I + i[1]]) for i in diff[:4]]
    got, want = (O.dequantise(c, scales) for c in (A.cpu().numpy(), codes))
    assert np.array_equal(got, want)                             # signs too (of zeros aside)
    for half, v in ((0, hd[:, :I]), (1, hd[:, I:])):
        c, s = O.quantise(v, True)
        assert np.array_equal(sH[:, half].cpu().numpy(), s)
        assert np.array_equal(Hq[:, half * I:(half + 1) * I].cpu().numpy(), c)
    assert torch.equal(A, A2) and torch.equal(sA, sA2) and none is None and none2 is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_far_gates(dtype):
    """Gates up to the type's largest number, on both sides, forward and backward."""
    rng = np.random.default_rng(5)
    far = np.array([3.3e38, 2.4e38, 1e30, 1e4, 151, 149, 120, 100, 89, 87, 81, 80, 79])
    g = rng.choice(np.concatenate([far, -far]), (26, 256))
    u = rng.standard_normal(g.shape) * np.minimum(1, 1e3 / np.abs(g))
    g[::2], u[::2] = np.concatenate([far, -far])[:, None][::2], rng.standard_normal((13, 256)) * 1e-3
    h = torch.from_numpy(np.concatenate([g, u], 1)).to(DTYPE[dtype]).to(DEV)
    A, sA, Hq, sH = dg.swiglu_fp8(h)
    torch.cuda.synchronize()
    hd = h.double().cpu().numpy()
    with np.errstate(over="ignore"):
        codes, scales = O.quantise(O.swiglu(hd[:, :256], hd[:, 256:]), True)
    assert np.array_equal(sA.cpu().numpy(), scales)
    assert np.array_equal(A.cpu().numpy() & 0x7F, codes & 0x7F)
    da = torch.from_numpy(rng.standard_normal(g.shape)).to(DTYPE[dtype]).to(DEV)
    dH = dg.swiglu_fp8_bwd(da, Hq, sH)
    gd, ud = (O.dequantise(Hq[:, i * 256:(i + 1) * 256].cpu().numpy(), sH[:, i].cpu().numpy()) for i in (0, 1))
    with np.errstate(over="ignore"):
        dg_, du, mass = O.swiglu_bwd(da.double().cpu().numpy(), gd, ud)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    for got, want, m in ((dH[:, :256], dg_, mass), (dH[:, 256:], du, np.abs(du))):
        bound = half * np.abs(want) + 2.0 ** -20 * m + 2.0 ** -100 * np.maximum(1, np.abs(gd))
        ok = np.abs(got.double().cpu().numpy() - want) <= bound
        # beyond the type's largest number the result is infinite
        top = float(torch.finfo(DTYPE[dtype]).max)
        ok |= (np.abs(want) > top * (1 - 2.0 ** -8)) & np.isinf(got.double().cpu().numpy())
        assert ok.all(), np.argwhere(~ok)[:4]


def test_swiglu_many_values():
    """A million ordinary values: none lands on the wrong side of a border."""
    rng = np.random.default_rng(0)
    h = torch.from_numpy(rng.standard_normal((256, 8192)) * 2).to(torch.bfloat16).to(DEV)
    A, sA, _, _ = dg.swiglu_fp8(h)
    hd = h.double()
    a = hd[:, 4096:] * (hd[:, :4096] / (1 + torch.exp(-hd[:, :4096])))
    amax = a.abs().view(256, 32, 128).amax(2)
    s = sA.double()
    assert bool(((amax <= 448 * s) & (amax > 224 * s)).all())
    v = (a.view(256, 32, 128) / s[:, :, None]).view(256, 4096).cpu().numpy()
    from oracle import encode_nearest
    assert np.array_equal(A.cpu().numpy(), encode_nearest(v))


def test_swiglu_not_finite_values_stay_in_their_block():
    """Codes of a block with infinities or NaN are unspecified; other blocks' are not."""
    h = torch.randn(3, 2 * 256, device=DEV)
    clean = dg.swiglu_fp8(h)
    h[1, 5], h[1, 256 + 9], h[1, 17] = float("inf"), float("nan"), -float("inf")
    got = dg.swiglu_fp8(h)
    torch.cuda.synchronize()
    for c, d in zip(clean, got):
        assert torch.equal(c[0], d[0]) and torch.equal(c[2], d[2])
    assert torch.equal(clean[0][1, 128:], got[0][1, 128:]) and torch.equal(clean[2][1, 128:256], got[2][1, 128:256])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,I", [(1, 16), (17, 128), (33, 176), (40, 1424)])
def test_swiglu_bwd(M, I, dtype):
    log(f"swiglu_bwd M={M} I={I} {dtype}")
    rng = np.random.default_rng(M * I)
    g = rng.standard_normal((M, I)) * np.exp2(rng.uniform(-3, 5, (M, 1)))       # up to about +-100
    u = rng.standard_normal((M, I))
    g[0] = 0
    h = torch.from_numpy(np.concatenate([g, u], 1)).to(torch.bfloat16).to(DEV)
    _, _, Hq, sH = dg.swiglu_fp8(h)
    da = torch.from_numpy(rng.standard_normal((M, I))).to(DTYPE[dtype]).to(DEV)
    dH = dg.swiglu_fp8_bwd(da, Hq, sH)
    torch.cuda.synchronize()
    gd = O.dequantise(Hq[:, :I].cpu().numpy(), sH[:, 0].cpu().numpy())
    ud = O.dequantise(Hq[:, I:].cpu().numpy(), sH[:, 1].cpu().numpy())
    dg_, du, mass = O.swiglu_bwd(da.double().cpu().numpy(), gd, ud)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    for got, want, m in ((dH[:, :I], dg_, mass), (dH[:, I:], du, np.abs(du))):
        # 2^-100: gates below -80 count as -80, and BF16 results may be subnormal
        bound = half * np.abs(want) + 2.0 ** -20 * m + 2.0 ** -100
        err = np.abs(got.double().cpu().numpy() - want)
        assert np.all(err <= bound), float((err / bound).max())


def wgrad_data(counts, align, N, K, seed, pow2=True):
    """Operands with NaN (dY, scales) and the NaN code (X) in rows of padding."""
    rng = np.random.default_rng(seed)
    G = len(counts)
    seg = [-(-c // align) * align for c in counts]
    offs = np.concatenate([[0], np.cumsum(seg)]).astype(np.int32)
    M = int(offs[-1])
    real = np.zeros(M, bool)
    for e in range(G):
        real[offs[e]:offs[e] + counts[e]] = True
    x = rng.standard_normal((M, K)) * np.exp2(rng.uniform(-4, 4, (M, 1)))
    codes, scales = O.quantise(x, pow2) if M else (np.zeros((0, K), np.uint8), np.zeros((0, -(-K // 128)), np.float32))
    codes[~real], scales[~real] = 0x7F, np.nan
    dy = torch.from_numpy(rng.standard_normal((M, N)) * 0.1).to(torch.bfloat16)
    dy[torch.from_numpy(~real)] = float("nan")
    return offs, np.array(counts, np.int32), M, codes, scales, dy


def to_dev(*a):
    return [torch.from_numpy(np.ascontiguousarray(v)).to(DEV) if isinstance(v, np.ndarray) else v.to(DEV) for v in a]


def check_wgrad(got, want, mass, counts, out, extra=0.0):
    n = np.array(counts).reshape(-1, 1, 1) + 1
    bound = n * 2.0 ** -23 * mass + extra * mass
    bound = bound + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * (np.abs(want) + bound)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())


WGRAD = [([1], 1, 8, 16), ([5], 128, 128, 128), ([0, 33, 1, 0, 64], 1, 136, 144), ([128, 0, 129, 31], 128, 264, 272),
         ([300, 7], 128, 520, 48), ([0, 0], 1, 24, 32), ([257], 1, 256, 512), ([70, 500, 2], 128, 384, 256)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,align,N,K", WGRAD)
def test_wgrad(counts, align, N, K, out):
    log(f"wgrad counts={counts} align={align} N={N} K={K} {out}")
    offs, cnt, M, codes, scales, dy = wgrad_data(counts, align, N, K, seed=N + K)
    want, mass = O.wgrad(np.nan_to_num(dy.float().numpy()), np.nan_to_num(O.dequantise(codes, scales)), offs, cnt)
    d = to_dev(dy, codes, scales, offs, cnt)
    dW = torch.full((len(counts), N, K), float("nan"), dtype=DTYPE[out], device=DEV)
    dg.grouped_wgrad_fp8(d[0], d[1], d[2], d[3], d[4], out_dtype=out, dW=dW)
    torch.cuda.synchronize()
    check_wgrad(dW, want, mass, counts, out)
    again = dg.grouped_wgrad_fp8(*d, out_dtype=out)
    assert torch.equal(again, dW)                                # bitwise repeatable


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("G,N,K", [(260, 136, 144), (65, 520, 272), (3, 2056, 1552)])
def test_wgrad_many_tiles(G, N, K, out):
    """More tiles than CUs, the last of each row and column partial."""
    log(f"wgrad G={G} N={N} K={K} {out}")
    counts = np.random.default_rng(G).integers(0, 140, G).tolist()
    counts[0] = 0
    offs, cnt, M, codes, scales, dy = wgrad_data(counts, 1, N, K, seed=G)
    d = to_dev(dy, codes, scales, offs, cnt)
    got = dg.grouped_wgrad_fp8(*d, out_dtype=out)
    x, y = (torch.from_numpy(v) for v in (O.dequantise(codes, scales), dy.double().numpy()))
    want = torch.stack([y[o:o + n].T @ x[o:o + n] for o, n in zip(offs, cnt)]).numpy()
    mass = torch.stack([y[o:o + n].abs().T @ x[o:o + n].abs() for o, n in zip(offs, cnt)]).numpy()
    check_wgrad(got, want, mass, counts, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_wgrad_accumulates(out):
    counts = [40, 0, 65]
    offs, cnt, M, codes, scales, dy = wgrad_data(counts, 1, 72, 160, seed=1)
    want, mass = O.wgrad(dy.float().numpy(), O.dequantise(codes, scales), offs, cnt)
    dW = torch.randn(3, 72, 160, device=DEV).to(DTYPE[out])
    base = dW.double().cpu().numpy()
    dg.grouped_wgrad_fp8(*to_dev(dy, codes, scales, offs, cnt), out_dtype=out, dW=dW, accumulate=True)
    check_wgrad(dW, base + want, np.abs(base) + mass, counts, out)
    assert np.array_equal(dW[1].double().cpu().numpy(), base[1])


def test_wgrad_without_counts_takes_whole_segments():
    offs, cnt, M, codes, scales, dy = wgrad_data([96, 130, 10], 1, 40, 64, seed=2)
    d = to_dev(dy, codes, scales, offs, cnt)
    assert torch.equal(dg.grouped_wgrad_fp8(*d[:4]), dg.grouped_wgrad_fp8(*d))


def test_wgrad_other_scales_round_the_activation_once():
    """amax / 448 scales: S dec(Q) enters the product rounded to BF16, half a step."""
    counts = [100, 30]
    offs, cnt, M, codes, scales, dy = wgrad_data(counts, 1, 64, 256, seed=3, pow2=False)
    want, mass = O.wgrad(dy.float().numpy(), O.dequantise(codes, scales), offs, cnt)
    got = dg.grouped_wgrad_fp8(*to_dev(dy, codes, scales, offs, cnt))
    # the FP32 product S dec(Q) rounds once, then BF16
    check_wgrad(got, want, mass, counts, "f32", extra=2.0 ** -8 + 2.0 ** -23)


def test_wgrad_long_expert():
    """One expert with many rows: the sums stay within FP32's."""
    offs, cnt, M, codes, scales, dy = wgrad_data([20000], 1, 64, 128, seed=4)
    x = O.dequantise(codes, scales)
    want = dy.double().numpy().T @ x
    got = dg.grouped_wgrad_fp8(*to_dev(dy, codes, scales, offs, cnt))
    rel = np.linalg.norm(got[0].double().cpu().numpy() - want) / np.linalg.norm(want)
    # random signs: sums of n terms have a norm of sqrt(n) of them, errors of n roundings sqrt(n) 2^-24 of the
    # running sum's size; 20000 rows in steps of 16 or more
    assert rel <= np.sqrt(20000 / 16) * 2.0 ** -23


def test_wgrad_is_deaf_to_the_order_of_experts():
    """The same rows at another place in the matrix give the same bits."""
    offs, cnt, M, codes, scales, dy = wgrad_data([50, 90], 1, 128, 128, seed=5)
    d = to_dev(dy, codes, scales, offs, cnt)
    both = dg.grouped_wgrad_fp8(*d)
    alone = dg.grouped_wgrad_fp8(d[0][50:].contiguous(), d[1][50:].contiguous(), d[2][50:].contiguous(),
                                 torch.tensor([0, 90], dtype=torch.int32, device=DEV))
    assert torch.equal(both[1], alone[0])


def test_rows_past_32_bit_offsets():
    """Operands and results whose byte offsets pass 2^32."""
    M, I = 70001, 32768
    h = torch.zeros(M, 2 * I, device=DEV, dtype=torch.bfloat16)
    last = torch.randn(3, 2 * I, device=DEV).bfloat16()
    h[-3:] = last
    A, sA, Hq, sH = dg.swiglu_fp8(h)
    want = dg.swiglu_fp8(last)
    for got, w in zip((A, sA, Hq, sH), want):
        assert torch.equal(got[-3:], w)
    assert not A[:-3].any() and bool((sA[:-3] == 1).all())
    da = torch.randn(3, I, device=DEV).bfloat16()
    dA = h[:, :I].contiguous()
    dA[-3:] = da
    dH = dg.swiglu_fp8_bwd(dA, Hq, sH)
    assert torch.equal(dH[-3:], dg.swiglu_fp8_bwd(da, want[2], want[3]))
    del h, dA, A, Hq
    # dY = dH: 2 I columns
    x = torch.randint(0, 0x70, (M, 16), dtype=torch.uint8, device=DEV)
    s = torch.ones(M, 1, device=DEV)
    offs = torch.tensor([0, M - 3, M], dtype=torch.int32, device=DEV)
    counts = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    dW = dg.grouped_wgrad_fp8(dH, x, s, offs, counts)
    alone = dg.grouped_wgrad_fp8(dH[-3:].contiguous(), x[-3:].contiguous(), s[-3:].contiguous(),
                                 torch.tensor([0, 3], dtype=torch.int32, device=DEV))
    assert torch.equal(dW[1], alone[0]) and not dW[0].any()


def test_results_past_32_bit_offsets():
    """The last of many experts' weight gradients lies past 2^32 bytes."""
    G, N, K = 70, 4096, 4096
    dy, x = torch.randn(G, N, device=DEV).bfloat16(), torch.randint(0, 0x70, (G, K), dtype=torch.uint8, device=DEV)
    s = torch.ones(G, K // 128, device=DEV)
    offs = torch.arange(G + 1, dtype=torch.int32, device=DEV)
    dW = dg.grouped_wgrad_fp8(dy, x, s, offs)
    assert dW.numel() * 4 > 1 << 32
    xv = x.view(torch.float8_e4m3fn).float()
    for e in (0, G - 2, G - 1):                                  # single products, exact in FP32
        assert torch.equal(dW[e], dy[e].float()[:, None] * xv[e][None])


def test_refusals():
    z = torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError):
        dg.swiglu_fp8(z[:, :63].contiguous())
    with pytest.raises(dg.DGError):
        dg.swiglu_fp8(z[:, :40].contiguous())
    A, sA, Hq, sH = dg.swiglu_fp8(z)
    with pytest.raises(ValueError):
        dg.swiglu_fp8_bwd(z[:, :32].contiguous(), Hq[:, :48].contiguous(), sH)
    offs = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        dg.grouped_wgrad_fp8(z, A, sA, offs)                     # float32 gradients
    with pytest.raises(ValueError):
        dg.grouped_wgrad_fp8(z.bfloat16(), A, sA, offs, accumulate=True)
    with pytest.raises(dg.DGError):
        dg.grouped_wgrad_fp8(z[:, :20].bfloat16().contiguous(), A, sA, offs)
