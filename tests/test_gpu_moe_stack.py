"""The operators around a block put together (examples/moe_layer.py): a stack of
mixture-of-experts blocks, every stage of its forward and backward pass against the
float64 oracle on the stage's own inputs, under graph capture, and decode.  Needs a GPU.

Tolerances are those of the stages' own tests: a norm's FP32 sums and products within
(8 + 18) u (R') and 48 u (N) of the magnitudes, u = 2^-24, and half a step of BF16; the
gradients within 128 u (stream) and 256 u (block), sums over T rows a rounding a row and
520 more; the router's weights within 100 u for logits of a range below 18."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import block as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
BF16 = 2.0 ** -8
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def n(t):
    return (t.double() if t.is_floating_point() else t).cpu().numpy()


def setup(example, T=150, blocks=2, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    stack = example.MoEStack(blocks, 6, 2, 256, 384, generator=g, balance=0.5)
    for b in stack.blocks:                                    # not all ones
        for p in (b.w_pre, b.w_post, b.gate):
            p.add_(torch.randn(256, device=DEV, generator=g) * 0.2)
    x = torch.randn(T, 256, device=DEV, generator=g).bfloat16()
    dout = torch.randn(T, 256, device=DEV, generator=g).bfloat16()
    return stack, x, dout


def close(got, want, bound, what):
    off = np.abs(n(got) - want)
    assert got.shape == want.shape and (off <= bound).all(), (what, float((off - bound).max()))


def test_stage_by_stage(example):
    stack, x, dout = setup(example)
    T = len(x)
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    mask[140:] = False
    out, losses, (_, saved) = stack.forward(x, mask)
    torch.cuda.synchronize()
    norms = [b.w_pre for b in stack.blocks] + [stack.w_last]
    stream, R = x, n(x)
    N = O.residual_norm(R, w_pre=n(norms[0]), eps=EPS)[1]
    close(saved[0][0], N, 48 * U * np.abs(N) + BF16 * np.abs(N), "first norm")
    alpha = float(np.float32(stack.alpha))
    for i, b in enumerate(stack.blocks):
        tokens, logits, r, y, of_layer, after = saved[i]
        ids, w, counts, sums, routed, loss = O.route(n(logits), 2, False, True, 1.0, mask=n(mask))
        assert np.array_equal(n(r.ids), ids) and np.array_equal(n(r.counts), counts) and int(r.routed) == routed == 140
        assert np.ptp(n(logits)) < 18
        close(r.weights, w, 100 * U * w, "weights")
        assert abs(float(losses[i]) - loss) <= 400 * U * loss
        assert not n(y)[140:].any()                           # rows without a token get nothing
        stage = [n(stream), n(y), n(b.w_post), n(b.gate), alpha, n(norms[i + 1]), EPS]
        want, N, z = O.residual_norm(*stage)
        mass = np.abs(stage[0]) + np.abs(z)
        close(after, want, 26 * U * mass + BF16 * np.abs(want), "stream")
        got = out if i + 1 == len(stack.blocks) else saved[i + 1][0]
        close(got, N, 48 * U * mass * O.rstd(want, EPS) * np.abs(stage[5]) + BF16 * np.abs(N), "norm")
        stream = after


def test_backward_stage_by_stage(example, monkeypatch):
    """Every call of the two backward operators within a step, on the inputs it got, and
    that their results are what the step returns."""
    stack, x, dout = setup(example)
    _, _, state = stack.forward(x)
    calls = []

    def watched(name):
        f = getattr(dg, name)

        def call(*args, **kw):
            r = f(*args, **kw)
            calls.append((name, args, kw, r))
            return r
        monkeypatch.setattr(dg, name, call)

    watched("residual_norm_bwd")
    watched("moe_route_bwd")
    dx, grads = stack.backward(dout, state)
    torch.cuda.synchronize()
    assert [c[0] for c in calls] == ["residual_norm_bwd", "moe_route_bwd"] * 2 + ["residual_norm_bwd"]
    T = len(x)
    rows = (T + 520) * U
    for name, args, kw, r in calls:
        if name == "moe_route_bwd":
            dw, logits, ids = args
            want, mass = O.route_bwd(n(dw), n(logits), n(ids), False, True, 1.0, float(kw["dloss"]), n(kw["counts"]),
                                     int(kw["routed"]))
            close(r, want, 400 * U * mass + U * np.abs(want), "logits")
            continue
        dR, dN, R = args[:3]
        Y = args[3] if len(args) > 3 else None
        opt = lambda k: None if kw.get(k) is None else n(kw[k])
        want = O.residual_norm_bwd(None if dR is None else n(dR), n(dN), n(R), None if Y is None else n(Y), opt("w_post"),
                                   opt("gate"), float(np.float32(kw.get("alpha", 1.0))), opt("w_pre"), EPS)
        for key, c in (("dR", 128 * U), ("dY", 256 * U), ("dw_post", 256 * U + rows), ("dgate", 256 * U + rows),
                       ("dw_pre", 128 * U + rows)):
            got = getattr(r, key)
            assert (got is None) == (key not in want)
            if got is not None:
                w, mass = want[key]
                close(got, w, c * mass + (BF16 if got.dtype == torch.bfloat16 else U) * np.abs(w), key)
    assert torch.equal(dx, calls[-1][3].dR)
    shapes = [p.shape for p in stack.parameters]
    assert [d.shape for d in grads] == shapes and all(bool(torch.isfinite(d).all()) for d in grads)
    per = len(stack.blocks[0].parameters)
    last, first = calls[0][3], calls[2][3]
    assert torch.equal(grads[per + 2], last.dw_post) and torch.equal(grads[per + 3], last.dgate)
    assert torch.equal(grads[2], first.dw_post) and torch.equal(grads[3], first.dgate)
    assert torch.equal(grads[0], calls[4][3].dw_pre) and torch.equal(grads[per], first.dw_pre)
    assert torch.equal(grads[-1], last.dw_pre)


def test_update_clips(example):
    stack, x, dout = setup(example)
    _, grads = stack.backward(dout, stack.forward(x)[2])
    before, params = [n(d) for d in grads], [n(p) for p in stack.parameters]
    norm, factor = O.clip(before, 0.25)
    assert factor < 1
    got = stack.update(grads, 0.5, 0.25)
    torch.cuda.synchronize()
    assert abs(float(got.double()) - norm) <= 2 * U * norm
    for d, b, p, q in zip(grads, before, stack.parameters, params):
        assert (np.abs(n(d) - b * factor) <= 4 * U * np.abs(b * factor) + 2.0 ** -140).all()
        want = q - 0.5 * b * factor
        assert (np.abs(n(p) - want) <= 2 * U * np.abs(want) + 4 * U * np.abs(b * factor) + 2.0 ** -140).all()


def test_step_under_graph_capture(example):
    """Forward, backward, norm and clipping captured once and replayed on other inputs,
    with eager steps between the replays."""
    stack, x, dout = setup(example, T=300)
    out = None

    def step():
        y, losses, saved = stack.forward(x)
        dx, grads = stack.backward(dout, saved)
        norm = dg.grad_norm(grads)
        clipped = dg.clip_grads(grads, norm, 0.5, out=[torch.empty_like(d) for d in grads])
        return (y, *losses, dx, norm, *clipped)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                # the stream's workspace exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in range(4):
        _, x2, d2 = setup(example, T=300, seed=seed + 1)
        x.copy_(x2)
        dout.copy_(d2)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (seed, i)


def test_two_streams_at_once():
    """The operators that take workspaces, on two streams: each as alone."""
    T, E, H = 6000, 256, 1408
    made = []
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        made.append([torch.randn(T, E, generator=g).cuda(), (torch.randn(E, generator=g) * 0.1).cuda()] +
                    [torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(4)] +
                    [torch.randn(H, generator=g).cuda() for _ in range(2)] + [torch.randn(300000, generator=g).cuda()])

    def run(logits, bias, dr, dn, r, y, wa, wb, grad):
        route = dg.moe_route(logits, 8, score="sigmoid", bias=bias)
        dlogits = dg.moe_route_bwd(route.weights, logits, route.ids, score="sigmoid", dloss=route.loss,
                                   counts=route.counts, routed=route.routed)
        norms = dg.residual_norm_bwd(dr, dn, r, y, w_post=wa, w_pre=wb)
        norm = dg.grad_norm([grad, wa])
        clipped = dg.clip_grads([grad], norm, 1.0, out=[torch.empty_like(grad)])
        return [t for t in (*route, dlogits, *norms, norm, *clipped) if t is not None]

    alone = []
    for m in made:
        alone.append(run(*m))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*made[i]))
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for one in runs:
            assert len(one) == len(want) and all(torch.equal(p, q) for p, q in zip(one, want))


@pytest.mark.parametrize("T", [1, 5])
def test_decode(example, T):
    """Roundings of the products in another order move codes by a step here and there,
    2^-3 of a value: far below a wrong route or norm."""
    stack, x, _ = setup(example, T=T)
    got, want = stack.decode(x), stack.forward(x)[0]
    assert float((got.double() - want.double()).norm() / want.double().norm()) <= 2.0 ** -5


@pytest.mark.parametrize("blocks", [0, 2])
def test_example_runs(example, monkeypatch, capsys, blocks):
    monkeypatch.setattr(sys, "argv", ["moe_layer.py", "--experts", "4", "--hidden", "256", "--inner", "256", "--tokens",
                                      "200", "--steps", "2", "--blocks", str(blocks)])
    example.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 3 and "decode" in lines[-1]
