"""The norm of many gradients and their clipping against the float64 oracle.  Needs a GPU.

Tolerances: squares and sums are in 64 bits, so the norm is within its one rounding,
2^-24, of the value (and 2^-40 for the sums); the factor rounds once more and the product
once, then the output's type: 3 x 2^-24 and half a step."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import block as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def make(shapes, dtypes, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * size).to(d).to(DEV) for s, d in zip(shapes, dtypes)]


def n(t):
    return t.double().cpu().numpy()


def check(grads, max_norm, out=None, stream=None):
    before = [n(t) for t in grads]
    norm, factor = O.clip(before, max_norm)
    got = dg.grad_norm(grads, stream=stream)
    back = dg.clip_grads(grads, got, max_norm, out=out, stream=stream)
    torch.cuda.synchronize()
    assert got.dim() == 0 and got.dtype == F and abs(float(got.double()) - norm) <= (U + 2.0 ** -40) * norm
    assert back is (grads if out is None else out)
    for t, b in zip(back, before):
        want = b * factor
        assert (np.abs(n(t) - want) <= (3 * U + HALF[t.dtype]) * np.abs(want) + 2.0 ** -140).all()
    if out is not None:
        for t, b in zip(grads, before):
            assert np.array_equal(n(t), b)
    return got


MANY = [(1,), (7,), (16384,), (16385,), (3, 5, 7), (0,), (40000,), (2, 8191), (130,), (1, 1, 1, 1)]


@pytest.mark.parametrize("max_norm", [1.0, 1e6])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("place", ["in place", "same", "f32", "bf16"])
def test_clip(max_norm, kind, place):
    types = {"f32": [F] * 10, "bf16": [B] * 10, "mixed": [F, B] * 5}[kind]
    grads = make(MANY, types)
    out = None
    if place != "in place":
        out = [torch.full_like(t, 9.0, dtype={"same": t.dtype, "f32": F, "bf16": B}[place]) for t in grads]
    check(grads, max_norm, out)


@pytest.mark.parametrize("count", [1, 95, 96, 97, 193, 500])
def test_clip_many_tensors(count):
    """More tensors than one launch takes; empty ones among them."""
    rng = np.random.default_rng(count)
    shapes = [(int(rng.integers(0, 300)),) for _ in range(count - 1)] + [(50000,)]
    check(make(shapes, [F if i % 3 else B for i in range(count)], count), 0.5)


def test_clip_views_at_any_element():
    """Tensors that lie at odd elements of larger ones, what is around them left as it was."""
    for dtype in (F, B):
        for at in range(9):
            whole = make([(70000,)], [dtype])[0]
            other = torch.zeros(70000, dtype=dtype, device=DEV)
            keep = whole.clone()
            g = [whole[at:at + 20001], whole[30001 + at:30001 + at + 17], whole[40008:60001]]
            out = [other[at + 1:at + 20002], other[30001:30018], other[40009:60002]]
            check(g, 1.0, out)
            assert torch.equal(whole, keep)
            edges = torch.ones(70000, dtype=torch.bool, device=DEV)
            for a, b in ((at + 1, at + 20002), (30001, 30018), (40009, 60002)):
                edges[a:b] = False
            assert not other[edges].any()
            check(g, 1.0)
            mine = torch.ones(70000, dtype=torch.bool, device=DEV)
            for a, b in ((at, at + 20001), (30001 + at, 30018 + at), (40008, 60001)):
                mine[a:b] = False
            assert torch.equal(whole[mine], keep[mine])


def test_norm_counts_a_tensor_twice_and_nothing():
    g = make([(100,)], [F])[0]
    once, twice = dg.grad_norm([g]), dg.grad_norm((g, g))
    assert abs(float(twice / once) - 2 ** 0.5) < 4 * U
    assert float(dg.grad_norm([g[:0]])) == 0
    z = torch.zeros(50, device=DEV)
    norm = dg.grad_norm([z])
    assert float(norm) == 0
    dg.clip_grads([z], norm, 1.0)
    assert not z.any()


def test_norm_of_far_sizes():
    """Squares that FP32 holds neither above nor below."""
    for size in (1e30, 1e-30):
        check(make([(5000,), (300,)], [F, B], size=size), size)


def test_norm_nan_and_infinity():
    g = make([(5000,), (64,)], [F, F])
    g[0][77] = float("inf")
    norm = dg.grad_norm(g)
    assert float(norm) == float("inf")
    dg.clip_grads(g, norm, 1.0)
    assert torch.isnan(g[0][77]) and int(torch.isnan(g[0]).sum()) == 1 and not g[1].any() and not g[0][:77].any()
    g = make([(5000,), (64,)], [F, F])
    g[1][3] = float("nan")
    norm = dg.grad_norm(g)
    assert torch.isnan(norm)
    dg.clip_grads(g, norm, 1.0)
    assert all(torch.isnan(t).all() for t in g)


def test_clip_at_the_border():
    """A norm of exactly max_norm changes nothing; a larger max_norm neither."""
    g = [torch.tensor([3.0, 4.0], device=DEV)]
    norm = dg.grad_norm(g)
    assert float(norm) == 5
    dg.clip_grads(g, norm, 5.0)
    assert g[0].tolist() == [3, 4]
    dg.clip_grads(g, norm, 2.5)
    assert g[0].tolist() == [1.5, 2]


def test_clip_large():
    """Offsets past 2^31 bytes, and more partial sums than the last step has threads."""
    g = [torch.ones(700_000_000, dtype=F, device=DEV), torch.ones(40_000_000, dtype=B, device=DEV)]
    norm = dg.grad_norm(g)
    want = (740_000_000) ** 0.5
    assert abs(float(norm.double()) - want) <= 2 * U * want
    dg.clip_grads(g, norm, 1.0)
    f = float(np.float32(1.0 / float(norm.double())))
    assert bool((g[0] == f).all()) and bool((g[1] == torch.tensor(f).bfloat16().to(DEV)).all())


def test_clip_versions_and_saved_tensors():
    """What is written counts as written."""
    x = torch.randn(10, device=DEV, requires_grad=True)
    y = (x * 2).exp()
    v = y._version
    dg.clip_grads([y.detach()], dg.grad_norm([y.detach()]), 1e-3)
    assert y._version > v
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_clip_repeatable_on_a_side_stream():
    g = make([(100000,), (3, 777)], [F, B])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = check([t.clone() for t in g], 1.0)
    c = [t.clone() for t in g]
    torch.cuda.synchronize()
    assert torch.equal(a, check(c, 1.0, stream=s))


def test_clip_graph():
    g = make(MANY, [F, B] * 5)
    out = [torch.zeros_like(t, dtype=F) for t in g]

    def step():
        norm = dg.grad_norm(g)
        dg.clip_grads(g, norm, 1.0, out=out)
        return norm

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    for seed in range(4):
        for t, u in zip(g, make(MANY, [F, B] * 5, seed + 1)):
            t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert torch.equal(norm, step())
        for a, b in zip(got, out):
            assert torch.equal(a, b)


def test_clip_refusals():
    g = make([(10,), (20,)], [F, B])
    norm = dg.grad_norm(g)
    for bad in (lambda: dg.clip_grads(g, norm, 1.0, out=g[:1]), lambda: dg.clip_grads(g, norm, 1.0, out=[g[0], g[0]]),
                lambda: dg.clip_grads(g, torch.ones(2, device=DEV), 1.0), lambda: dg.grad_norm([g[0][::2]])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dg.clip_grads(g, norm, 0.0), lambda: dg.clip_grads([g[0], g[0]], norm, 1.0),
                lambda: dg.clip_grads([g[0][:6], g[0][5:]], norm, 1.0)):
        with pytest.raises(dg.DGError):
            bad()
    with pytest.raises(TypeError):
        dg.clip_grads(g, norm.double(), 1.0)
