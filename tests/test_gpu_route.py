"""The router and its gradient against the float64 oracle.  Needs a GPU.

Tolerances, counted in u = 2^-24, the half step of FP32.  A score's exponential is
within 4 u and takes x - m rounded, which moves it by D u for a range D of the logits; a
reciprocal costs 2 u, every other operation u.  So a score is within (D + 12) u of
itself, its share in a sum of n of them within 2 (D + 12) u + (n's order of summation: at
most 22 additions one after another) u, and a weight with its scale 2 u more:
W = (2 D + 64) u bounds each of these with room for the gate 1 - s.  Sums of P over
tokens add, one after another, at most the turns of a workgroup, 2 of a wave, 16 waves
and 256 workgroups.  BF16 results add their half step, 2^-8.  What lies below FP32's
smallest normal number, 2^-126, is lost at any of these."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import block as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = 2.0 ** -120
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def logits(T, E, dtype, seed, kind="plain"):
    """A CPU tensor of router logits."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)
    if kind == "closed":
        x[torch.rand(T, E, generator=g) < 0.7] = -INF
        x[::5] = -INF
    elif kind == "ties":
        x = torch.round(x)
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "far":                                       # scores that underflow, but for their shares
        x = x * 20 - 300
    elif kind == "lowest":                                    # masked by the type's lowest value
        x[torch.rand(T, E, generator=g) < 0.5] = torch.finfo(dtype).min
        x[::4] = torch.finfo(dtype).min
    return x.to(dtype)


def n(t):
    return None if t is None else (t.double() if t.is_floating_point() else t).cpu().numpy()


def within(got, want, bound, what=""):
    got, want = n(got), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (what, float(off[bad].max()), np.argwhere(bad)[:4].tolist())


def weight_tolerance(x):
    """W: the range of the logits counts up to 110, past which scores are 0 in FP32."""
    f = x[np.isfinite(x)]
    return (2 * min(float(np.ptp(f)) if f.size else 0.0, 110.0) + 64) * U


def check(x, k, score, renorm, scale=1.0, bias=None, mask=None, balance=True, stream=None):
    xd = n(x)
    sigmoid = score == "sigmoid"
    dev = lambda t: None if t is None else t.to(DEV)
    r = dg.moe_route(dev(x), k, score=score, renormalise=renorm, scale=scale, bias=dev(bias), mask=dev(mask),
                     balance=balance, stream=stream)
    torch.cuda.synchronize()
    ids, w, counts, sums, routed, loss = O.route(xd, k, sigmoid, renorm, scale, n(bias), n(mask))
    assert r.ids.dtype == torch.int32 and np.array_equal(n(r.ids), ids)
    W = weight_tolerance(xd)
    within(r.weights, w, W * w + TINY, "weights")
    if not balance:
        assert r.counts is None and r.prob_sums is None and r.routed is None and r.loss is None
        return r, ids
    assert np.array_equal(n(r.counts), counts) and n(r.routed) == routed
    added = (len(xd) // 4096 + 2 + 2 + 16 + 256) * U
    within(r.prob_sums, sums, (W + added) * sums + len(xd) * TINY, "prob_sums")
    within(r.loss, loss, (W + added + 2 * U) * loss + TINY, "loss")
    assert r.loss.dim() == r.routed.dim() == 0
    return r, ids


SHAPES = [(1, 64, 2), (1, 1, 1), (5, 7, 7), (37, 60, 6), (130, 64, 2), (64, 65, 3), (33, 128, 8), (200, 256, 8),
          (65, 255, 16), (33, 257, 4), (19, 1000, 8), (17, 1024, 64), (9, 40, 33), (8, 300, 20), (3000, 16, 2)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(T, E, k, dtype, score):
    x = logits(T, E, dtype, seed=T + E)
    check(x, k, score, renorm=True, scale=2.5)
    check(x, k, score, renorm=False, balance=False)


@pytest.mark.parametrize("kind", ["closed", "ties", "equal", "far", "lowest"])
@pytest.mark.parametrize("E,k", [(12, 4), (100, 8), (400, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_hard_rows(kind, E, k, score, renorm):
    for dtype in (torch.float32, torch.bfloat16):
        check(logits(53, E, dtype, 3, kind), k, score, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["plain", "closed", "ties", "equal"])
@pytest.mark.parametrize("E,k", [(9, 3), (64, 4), (200, 8), (600, 10), (100, 20)])
def test_route_with_a_bias(score, kind, E, k):
    x = logits(301, E, torch.bfloat16, 4, kind)
    g = torch.Generator().manual_seed(5)
    zeros = torch.zeros(E)
    some = torch.randn(E, generator=g) * 0.1
    large = torch.randn(E, generator=g) * 300
    shut = some.clone()
    shut[::2] = -INF
    open_ = some.clone()
    open_[-1] = INF
    for bias in (zeros, some, large, shut, open_):
        check(x, k, score, True, bias=bias)
    check(x.float(), k, score, False, bias=some, balance=False)


def test_route_bias_that_tells_near_sums_apart():
    """Sums of score and bias that differ by far less than an FP32 step."""
    E, k, T = 64, 8, 64
    g = torch.Generator().manual_seed(6)
    x = torch.rand(T, E, generator=g) * 4
    s = 1 / (1 + torch.exp(-x[0].double()))
    bias = (0.75 - s).float()                                 # every sum within 2^-25 of 0.75
    x[:] = x[0]
    sums = s + bias.double()
    assert float(sums.max() - sums.min()) < 2.0 ** -24
    check(x, k, "sigmoid", True, bias=bias)


@pytest.mark.parametrize("E,k", [(64, 4), (256, 8), (1024, 8), (64, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_lowest_values_are_open(E, k, dtype):
    """The type's lowest value masks softly: chosen where nothing else is left, also as
    the last expert; only -inf closes."""
    x = torch.full((6, E), torch.finfo(dtype).min)
    x[1] = -INF
    x[1, E - 1] = torch.finfo(dtype).min
    x[2, : E - 2] = -INF
    x[3, 5] = 1.0
    x[4, E - 1] = torch.finfo(dtype).max
    x[5, ::2] = -torch.finfo(dtype).tiny
    r, ids = check(x.to(dtype), k, "softmax", True)
    assert ids[0].tolist() == list(range(k)) and ids[1, :2].tolist() == [E - 1, -1]
    check(x.to(dtype), k, "sigmoid", False, bias=torch.zeros(E))


@pytest.mark.parametrize("mask_type", [torch.bool, torch.uint8])
def test_route_mask(mask_type):
    x = logits(203, 60, torch.float32, 7, "closed")
    mask = (torch.rand(203, generator=torch.Generator().manual_seed(8)) < 0.6)
    x[~mask] = float("nan")                                   # rows without a token hold anything
    clean = torch.where(mask[:, None], x, torch.zeros(()))
    r = dg.moe_route(x.to(DEV), 6, mask=mask.to(mask_type).to(DEV))
    want, _ = check(clean, 6, "softmax", True, mask=mask)
    for a, b in zip(r, want):
        assert torch.equal(a, b)
    none = dg.moe_route(x.to(DEV), 6, mask=torch.zeros(203, dtype=mask_type, device=DEV))
    assert (none.ids == -1).all() and not none.weights.any() and not none.counts.any()
    assert int(none.routed) == 0 and float(none.loss) == 0 and not none.prob_sums.any()


def test_route_nothing():
    r = dg.moe_route(torch.zeros(0, 12, device=DEV), 3)
    assert r.ids.shape == (0, 3) and not r.counts.any() and not r.prob_sums.any()
    assert int(r.routed) == 0 and float(r.loss) == 0
    assert dg.moe_route(torch.zeros(0, 12, device=DEV), 3, balance=False).ids.shape == (0, 3)


@pytest.mark.parametrize("E", [10, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_nan_and_infinity(E, score, biased):
    """A row's NaN stays in the row, but for the sums; ids stay in range and distinct."""
    x = logits(20, E, torch.float32, 9)
    x[3, 4] = float("nan")
    x[7] = float("nan")
    x[11, 2] = INF
    bias = torch.zeros(E, device=DEV) if biased else None
    for renorm in (True, False):
        r = dg.moe_route(x.to(DEV), 5, score=score, renormalise=renorm, bias=bias)
        ids, w = n(r.ids), n(r.weights)
        assert ids.min() >= 0 and ids.max() < E and all(len(set(row)) == 5 for row in ids.tolist())
        assert np.isnan(w[7]).all()
        if score == "sigmoid" or not biased:                  # (softmax: all scores of the row are NaN)
            assert ids[3, 0] == 4 and np.isnan(w[3, 0]) and ids[11, 0] == 2
        assert np.isnan(w[11]).any() == (score == "softmax")
        assert np.isnan(n(r.prob_sums)).any() and np.isnan(n(r.loss))
        rows = [t for t in range(20) if t not in (3, 7, 11)]
        alone = dg.moe_route(x[rows].to(DEV), 5, score=score, renormalise=renorm, bias=bias)
        assert np.array_equal(ids[rows], n(alone.ids)) and np.array_equal(w[rows], n(alone.weights))


def test_route_many_tokens_one_expert():
    """More turns of every workgroup than one, all tokens to the same experts."""
    T, E, k = 40000, 24, 2
    x = torch.zeros(T, E)
    x[:, 5], x[:, 20] = 4, 3
    r, _ = check(x, k, "softmax", True)
    assert n(r.counts)[[5, 20]].tolist() == [T, T]


def test_route_more_tokens_than_a_grid_takes_at_once():
    """Millions of tokens: every workgroup in several turns also without the load."""
    T, E = 4_400_000, 4
    x = torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    want = x.argmax(1).int()
    a = dg.moe_route(x, 1, balance=False)
    b = dg.moe_route(x, 1)
    assert torch.equal(a.ids[:, 0], want) and torch.equal(b.ids[:, 0], want) and int(b.routed) == T
    assert torch.equal(b.counts.long(), torch.bincount(want, minlength=E)) and bool((a.weights == 1).all())
    dx = dg.moe_route_bwd(torch.ones(T, 1, device=DEV), x, a.ids, renormalise=False)
    last = dg.moe_route_bwd(torch.ones(5, 1, device=DEV), x[-5:].contiguous(), a.ids[-5:].contiguous(), renormalise=False)
    assert torch.equal(dx[-5:], last)


def test_route_repeatable_and_on_a_side_stream():
    x = logits(5000, 200, torch.float32, 10)
    a, _ = check(x, 8, "sigmoid", True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = check(x, 8, "sigmoid", True, stream=s)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


# ---------------------------------------------------------------- gradient

def check_bwd(x, ids, score, renorm, loss, seed=0, scale=1.5, counts=None, routed=None):
    g = torch.Generator().manual_seed(seed)
    T, E = x.shape
    dw = torch.randn(ids.shape, generator=g)
    there = (ids >= 0) & (ids < E)
    clean = np.where(there, ids, -1)
    if loss:
        counts = np.bincount(clean[clean >= 0], minlength=E) if counts is None else counts
        routed = int((clean >= 0).any(1).sum()) if routed is None else routed
        # scaled so that both parts are seen
        dloss = torch.tensor(float(max(1, routed)), dtype=torch.float32)
    else:
        dloss = None
    dev = lambda a, t: torch.as_tensor(np.ascontiguousarray(a)).to(t).to(DEV)
    args = dict(score=score, renormalise=renorm, scale=scale)
    if loss:
        args.update(dloss=dloss.to(DEV), counts=dev(counts, torch.int32), routed=dev(np.array(routed), torch.int32))
    dx = dg.moe_route_bwd(dw.to(DEV), x.to(DEV), dev(ids, torch.int32), **args)
    torch.cuda.synchronize()
    assert dx.dtype == x.dtype
    more = (float(dloss), counts, routed) if loss else ()
    xd = n(x)
    want, mass = O.route_bwd(n(dw), xd, clean, score == "sigmoid", renorm, scale, *more)
    # the sums over chosen experts and over all (at most 22 one after another) twice
    c = 2 * weight_tolerance(np.where((clean >= 0).any(1)[:, None], xd, 0.0)) + (ids.shape[1] + 64) * U
    within(dx, want, c * mass + HALF[x.dtype] * np.abs(want) + TINY * (1 + np.abs(mass).max()), "dx")
    return dx


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_bwd(T, E, k, score, renorm):
    for dtype in (torch.float32, torch.bfloat16):
        x = logits(T, E, dtype, T + E)
        ids = O.choose(n(x), k, False)
        for loss in (True, False):
            check_bwd(x, ids, score, renorm, loss)


@pytest.mark.parametrize("kind", ["closed", "ties", "equal", "far", "lowest"])
@pytest.mark.parametrize("E,k", [(12, 4), (100, 8), (400, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bwd_hard_rows(kind, E, k, score):
    for renorm in (True, False):
        x = logits(53, E, torch.float32, 3, kind)
        ids = O.choose(n(x), k, False, mask=np.arange(53) % 7 != 0)
        check_bwd(x, ids, score, renorm, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_bwd_ids_of_any_kind(score, renorm):
    """The same expert twice in a row, experts out of range, and rows without one."""
    x = logits(40, 30, torch.float32, 11)
    ids = np.random.default_rng(12).integers(-3, 34, (40, 5))
    ids[4] = 7
    ids[9] = -1
    ids[10] = [40, 30, -9, 2 ** 31 - 1, -2 ** 31]
    dx = check_bwd(x, ids, score, renorm, True)
    assert not n(dx)[[9, 10]].any()


def test_route_bwd_experts_that_are_closed():
    """Choices whose logits are -inf have no gradient, and no NaN."""
    x = torch.zeros(3, 6)
    x[0, 2] = -INF
    x[1] = -INF
    ids = torch.tensor([[2, 1], [0, 1], [3, 4]], dtype=torch.int32, device=DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dx = dg.moe_route_bwd(torch.ones(3, 2, device=DEV) + torch.arange(2, device=DEV), x.to(DEV), ids, score=score,
                                  renormalise=renorm, dloss=torch.ones((), device=DEV),
                                  counts=torch.ones(6, dtype=torch.int32, device=DEV),
                                  routed=torch.full((), 3, dtype=torch.int32, device=DEV))
            assert torch.isfinite(dx).all() and not dx[1].any() and dx[0, 2] == 0


def test_route_bwd_rows_without_a_choice_are_not_read():
    x = logits(50, 16, torch.float32, 13)
    ids = torch.as_tensor(O.choose(n(x), 2, False)).int()
    ids[::3] = -1
    dirty = x.clone()
    dirty[::3] = float("nan")
    dw = torch.randn(50, 2)
    dw_dirty = dw.clone()
    dw_dirty[::3] = float("nan")
    a = dg.moe_route_bwd(dw.to(DEV), x.to(DEV), ids.to(DEV))
    b = dg.moe_route_bwd(dw_dirty.to(DEV), dirty.to(DEV), ids.to(DEV))
    assert torch.equal(a, b) and not a[::3].any()


def test_route_bwd_against_differences():
    """The gradient of what moe_route itself returns, the loss and the weights times dw in
    [0, 1), by central differences along a direction within +-1.  The values' sum is at
    most T k + 1 and within 68 u of itself (logits of a range of 2): 68 u (T k + 1) / h.
    A token's third derivative along the direction stays below 3/2: T h^2 / 4."""
    T, E, k, h = 64, 16, 2, 2.0 ** -5
    g = torch.Generator().manual_seed(14)
    # gaps that 2 h does not close
    x = torch.randn(T, E, generator=g).argsort(1).argsort(1).double() * 0.125 - 1
    d = torch.rand(T, E, generator=g).double() * 2 - 1
    dw = torch.rand(T, k, generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            f = lambda x_: dg.moe_route(x_.float().to(DEV), k, score=score, renormalise=renorm)
            r, hi, lo = f(x), f(x + h * d), f(x - h * d)
            assert torch.equal(hi.ids, r.ids) and torch.equal(lo.ids, r.ids)
            dx = dg.moe_route_bwd(dw.to(DEV), x.float().to(DEV), r.ids, score=score, renormalise=renorm,
                                  dloss=torch.full((), 1.0, device=DEV), counts=r.counts, routed=r.routed)
            got = float((dx.double().cpu() * d).sum())
            value = lambda r_: float((r_.weights.double().cpu() * dw).sum()) + float(r_.loss.double())
            want = (value(hi) - value(lo)) / (2 * h)
            assert abs(got - want) <= 68 * U * (T * k + 1) / h + T * h * h / 4, (score, renorm, got, want)


def test_route_refusals():
    x = torch.zeros(6, 8, device=DEV)
    r = dg.moe_route(x, 2)
    f = torch.zeros(6, 2, device=DEV)
    one = torch.ones((), device=DEV)
    for bad in (lambda: dg.moe_route(x.t(), 2), lambda: dg.moe_route(x[:, :4], 2),
                lambda: dg.moe_route(x, 2, bias=torch.zeros(7, device=DEV)),
                lambda: dg.moe_route(x, 2, mask=torch.ones(7, dtype=torch.bool, device=DEV)),
                lambda: dg.moe_route_bwd(f, x, r.ids, dloss=one),
                lambda: dg.moe_route_bwd(f, x, r.ids[:5]), lambda: dg.moe_route_bwd(f[:, :1], x, r.ids),
                lambda: dg.moe_route_bwd(f, x, r.ids, dloss=torch.ones(2, device=DEV), counts=r.counts, routed=r.routed),
                lambda: dg.moe_route_bwd(f, x, r.ids, dloss=one, counts=r.counts[:4], routed=r.routed)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dg.moe_route(x, 2, bias=torch.zeros(8, device=DEV, dtype=torch.float64)),
                lambda: dg.moe_route(x, 2, mask=torch.ones(6, device=DEV)),
                lambda: dg.moe_route_bwd(f, x, r.ids.long())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dg.moe_route(x, 9), lambda: dg.moe_route(x, 0), lambda: dg.moe_route(x, 2, scale=INF),
                lambda: dg.moe_route(torch.zeros(2, 1025, device=DEV), 2), lambda: dg.moe_route(torch.zeros(2, 100, device=DEV), 65),
                lambda: dg.moe_route(torch.zeros(2, 0, device=DEV), 1)):
        with pytest.raises(dg.DGError):
            bad()


def test_route_graph():
    """Captured once, replayed on other inputs, with eager calls between the replays."""
    x = torch.zeros(700, 64, device=DEV)
    dw = torch.randn(700, 4, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    dloss = torch.full((), 3.0, device=DEV)

    def step():
        r = dg.moe_route(x, 4, score="sigmoid", bias=bias)
        return (*r, dg.moe_route_bwd(dw, x, r.ids, score="sigmoid", dloss=dloss, counts=r.counts, routed=r.routed))

    bias = torch.zeros(64, device=DEV)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        x.copy_(logits(700, 64, torch.float32, seed).to(DEV))
        bias.copy_(torch.randn(64, generator=torch.Generator().manual_seed(seed)) * 0.1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
