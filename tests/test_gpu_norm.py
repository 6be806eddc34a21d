"""The residual stream past a block, the norms before and after it, and their gradients
against the float64 oracle.  Needs a GPU.

Tolerances, counted in u = 2^-24, the half step of FP32.  A row's sum has 8 terms a thread
one after another (once more for each 4096 columns that do not fit the registers, H /
4096), 6 steps of a wave and 16 waves: within 30 u + H / 4096 u of its terms' magnitudes.
The root halves that for squares, the reciprocal root costs 2 u and the mean 1: rstd is
within s = 18 u + H / 8192 u of itself.  Forward: what the block adds is a product of up
to five factors (6 u) with an rstd, the stream one more rounding, the norm three more and
another rstd: R' within 8 u + s of |R| + |z|, N within 12 u + 2 s of (|R| + |z|) rstd |w|,
each plus the half step of its type.  Codes are of values in 64 bits and equal the
oracle's.  Backward, by the magnitudes of the terms: dR takes rstd^3, a row's sum and up to
ten operations, G = 3 s + 30 u + H / 4096 u + 10 u; dY the same again; sums over T rows add
a rounding a row and 520 of groups and workgroups at most.  Below FP32's normal numbers
everything is lost."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import block as O
from oracle import moe as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = 2.0 ** -120
rstd_error = lambda H: (18 + H / 8192) * U
gradient_error = lambda H: 3 * rstd_error(H) + (40 + H / 4096) * U
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def n(t):
    return None if t is None else (t.double() if t.is_floating_point() else t).cpu().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def within(got, want, bound, what):
    got = n(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (what, float(off[bad].max()), np.argwhere(bad)[:4].tolist())


def problem(T, H, rt, dt, block=True, post=True, gate=None, pre=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    p = dict(R=torch.randn(T, H, generator=g).to(rt), Y=(torch.randn(T, H, generator=g) * 3).to(dt) if block else None,
             w_post=1 + 0.3 * torch.randn(H, generator=g) if block and post else None,
             w_pre=1 + 0.3 * torch.randn(H, generator=g) if pre else None, gate=None)
    if block and gate:
        p["gate"] = torch.randn(H if gate == "channel" else (T, 1), generator=g)
    return p


def check(p, alpha=1.0, eps=1e-6, values=True, codes=None, dtype=None, stream=None):
    out = dg.residual_norm(dev(p["R"]), dev(p["Y"]), w_post=dev(p["w_post"]), gate=dev(p["gate"]), alpha=alpha,
                           w_pre=dev(p["w_pre"]), eps=eps, values=values, codes=codes, dtype=dtype, stream=stream)
    torch.cuda.synchronize()
    d = {k: n(v) for k, v in p.items()}
    eps = float(np.float32(eps))
    alpha = float(np.float32(alpha))
    stream_, N, z = O.residual_norm(d["R"], d["Y"], d["w_post"], d["gate"], alpha, d["w_pre"], eps)
    mass = np.abs(d["R"]) + np.abs(z)
    s = rstd_error(d["R"].shape[1])
    if p["Y"] is None:
        assert out.R is None
    else:
        assert out.R.dtype == p["R"].dtype
        within(out.R, stream_, (8 * U + s) * mass + HALF[p["R"].dtype] * np.abs(stream_) + TINY, "R")
    if p["w_pre"] is None:
        assert out.N is None and out.Q is None and out.S is None
        return out
    if values:
        t = out.N.dtype
        assert t == (p["Y"].dtype if p["Y"] is not None else {None: B, "bf16": B, "f32": F}[dtype])
        within(out.N, N, (12 * U + 2 * s) * mass * O.rstd(stream_, eps) * np.abs(d["w_pre"]) + HALF[t] * np.abs(N) + TINY, "N")
    else:
        assert out.N is None
    if codes:
        q, scales = M.quantise(N, codes == "pow2")
        assert np.array_equal(out.S.cpu().numpy(), scales) and np.array_equal(n(out.Q), q)
    else:
        assert out.Q is None and out.S is None
    return out


SIZES = [(1, 1), (1, 2048), (3, 8), (5, 7), (2, 512), (7, 513), (33, 1424), (9, 2047), (4, 4096), (3, 8192), (2, 8193),
         (3, 8200), (2, 20000), (2, 16411)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("rt,dt", [(B, B), (F, F), (F, B), (B, F)])
def test_norm(T, H, rt, dt):
    check(problem(T, H, rt, dt), alpha=0.5)
    check(problem(T, H, rt, dt, gate="channel", pre=False))
    check(problem(T, H, rt, dt, block=False), dtype="f32" if dt == F else "bf16")


@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("H", [768, 770, 9000])
def test_norm_parts(gate, post, pre, H):
    check(problem(21, H, F, B, True, post, gate, pre), alpha=-0.25)


@pytest.mark.parametrize("T,H", [(1, 16), (1, 2048), (3, 128), (5, 144), (40, 1424), (7, 4096), (2, 8192), (2, 8208),
                                 (3, 20000)])
@pytest.mark.parametrize("codes", ["pow2", "amax"])
@pytest.mark.parametrize("rt,dt", [(B, B), (F, F), (F, B), (B, F)])
def test_norm_codes(T, H, codes, rt, dt):
    check(problem(T, H, rt, dt, gate="token"), codes=codes)
    check(problem(T, H, rt, dt, block=False), codes=codes, values=False)


def test_norm_codes_are_the_products_operand():
    """Codes and scales go straight into the dense product."""
    p = problem(40, 256, B, B)
    out = check(p, codes="pow2")
    w = torch.randn(128, 256, generator=torch.Generator().manual_seed(1)).to(DEV)
    wq, ws = dg.quantize_fp8_blockscaled(w, 128)
    c = dg.gemm_fp8_blockscaled(out.Q, out.S, wq, ws, "f32")
    want = out.N.float() @ w.t()
    # both operands rounded to 4 significant bits, 256 products: far looser than what a wrong scale or layout gives
    assert float((c - want).norm() / want.norm()) < 0.08


def test_norm_rows_of_zeros_and_far_sizes():
    """Zero rows are zeros; squares that FP32 cannot hold, and values so small that eps
    is all there is."""
    for H in (64, 300, 9000):
        p = problem(12, H, F, F)
        p["R"][0], p["Y"][0] = 0, 0
        p["Y"][1] = 0
        p["Y"][2] *= 1e30
        p["R"][3] *= 1e37
        p["R"][4] *= 1e-30
        p["Y"][4] *= 1e-30
        p["R"][5] *= 1e-40                                    # subnormal
        p["Y"][5] *= 1e-40
        out = check(p)
        assert not n(out.N)[0].any()
        q = dict(p, Y=None, w_post=None)
        check(q, dtype="f32")
        if H % 16 == 0:
            c = check(dict(p), codes="pow2")
            assert not n(c.Q)[0].any() and (n(c.S)[0] == 1).all()


def test_norm_eps_counts():
    check(problem(4, 96, F, F), eps=100.0)
    check(problem(4, 96, F, F), eps=1e-30)


def test_norm_nan_and_infinity_stay_in_their_row():
    p = problem(9, 200, F, F)
    clean = dg.residual_norm(*(dev(p[k]) for k in ("R", "Y")), w_post=dev(p["w_post"]), w_pre=dev(p["w_pre"]))
    p["Y"][2, 5], p["R"][4, 1], p["Y"][6, 0] = float("nan"), float("inf"), float("-inf")
    out = dg.residual_norm(*(dev(p[k]) for k in ("R", "Y")), w_post=dev(p["w_post"]), w_pre=dev(p["w_pre"]))
    rows = [0, 1, 3, 5, 7, 8]
    assert torch.equal(out.R[rows], clean.R[rows]) and torch.equal(out.N[rows], clean.N[rows])
    assert torch.isnan(out.N[2]).all() and torch.isnan(out.N[4, 1]) and torch.isnan(out.N[6]).any()


@pytest.mark.parametrize("T", [0, 1])
def test_norm_few_rows(T):
    p = problem(T, 48, B, B, gate="token")
    out = check(p, codes="pow2")
    assert out.N.shape == (T, 48) and out.S.shape == (T, 1)


def test_norm_many_rows():
    """More rows than workgroups: each takes several."""
    check(problem(9000, 136, B, B, gate="token"))
    check(problem(9000, 144, B, B, gate="token"), codes="amax")
    check(problem(700, 4096, B, B))


def test_norm_past_2_31_elements():
    """Rows far behind give what they give alone, forward and backward."""
    T, H = 1_050_000, 2056
    g = torch.Generator(device=DEV).manual_seed(1)
    R = torch.empty(T, H, dtype=B, device=DEV)
    Y = torch.empty(T, H, dtype=B, device=DEV)
    for at in range(0, T, 150_000):
        R[at:at + 150_000].normal_(generator=g)
        Y[at:at + 150_000].normal_(generator=g)
    w, gate = torch.rand(H, device=DEV, generator=g) + 0.5, torch.rand(T, 1, device=DEV, generator=g)
    rows = [0, 777_777, T - 2, T - 1]
    few = [t[rows].contiguous() for t in (R, Y, gate)]
    out = dg.residual_norm(R, Y, w_post=w, gate=gate, w_pre=w)
    alone = dg.residual_norm(few[0], few[1], w_post=w, gate=few[2], w_pre=w)
    assert torch.equal(out.R[rows], alone.R) and torch.equal(out.N[rows], alone.N)
    got = dg.residual_norm_bwd(R, Y, out.R, Y, w_post=w, gate=gate, w_pre=w)
    del out
    one = dg.residual_norm_bwd(few[0], few[1], alone.R, few[1], w_post=w, gate=few[2], w_pre=w)
    assert torch.equal(got.dR[rows], one.dR) and torch.equal(got.dY[rows], one.dY) and torch.equal(got.dgate[rows], one.dgate)


def test_norm_rows_of_one_column_to_the_last():
    """As many rows as there are workgroups several thousand times over."""
    T = 30_000_000
    x = torch.ones(T, 1, device=DEV)
    x[-1] = -3
    out = dg.residual_norm(x, w_pre=torch.full((1,), 2.0, device=DEV), dtype="f32")
    assert bool(((out.N[:-1] - 2).abs() < 1e-5).all()) and abs(float(out.N[-1]) + 2) < 1e-5


# ---------------------------------------------------------------- backward

def check_bwd(p, alpha=1.0, eps=1e-6, seed=3, with_dR=True, stream=None):
    g = torch.Generator().manual_seed(seed)
    T, H = p["R"].shape
    pre = p["w_pre"] is not None
    nt = p["Y"].dtype if p["Y"] is not None else B
    dR = torch.randn(T, H, generator=g).to(p["R"].dtype) if with_dR else None
    dN = torch.randn(T, H, generator=g).to(nt) if pre else None
    got = dg.residual_norm_bwd(dev(dR), dev(dN), dev(p["R"]), dev(p["Y"]), w_post=dev(p["w_post"]),
                               gate=dev(p["gate"]), alpha=alpha, w_pre=dev(p["w_pre"]), eps=eps, stream=stream)
    torch.cuda.synchronize()
    d = {k: n(v) for k, v in p.items()}
    want = O.residual_norm_bwd(n(dR), n(dN), d["R"], d["Y"], d["w_post"], d["gate"], float(np.float32(alpha)), d["w_pre"],
                               float(np.float32(eps)))
    types = dict(dR=p["R"].dtype, dY=nt, dw_post=F, dgate=F, dw_pre=F)
    g, rows = gradient_error(H), (T + 520) * U
    for name, c in (("dR", g), ("dY", 2 * g), ("dw_post", 2 * g + rows), ("dgate", 2 * g + rows), ("dw_pre", g + rows)):
        t = getattr(got, name)
        if name not in want:
            assert t is None, name
            continue
        w, mass = want[name]
        assert t.dtype == types[name]
        if t.numel():
            within(t, w, c * mass + HALF[t.dtype] * np.abs(w) + TINY * (1 + mass.max()), name)
    return got


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("rt,dt", [(B, B), (F, F), (F, B), (B, F)])
def test_norm_bwd(T, H, rt, dt):
    check_bwd(problem(T, H, rt, dt, gate="channel"), alpha=0.5)
    check_bwd(problem(T, H, rt, dt, gate="token", post=False), with_dR=False)


@pytest.mark.parametrize("T,H", [(257, 72), (511, 4096), (513, 4088), (600, 2048), (1009, 1408), (1000, 514), (2049, 264),
                                 (4096, 512), (4097, 511)])
@pytest.mark.parametrize("rt,dt", [(B, B), (F, F), (F, B)])
def test_norm_bwd_of_a_turn(T, H, rt, dt):
    """About as many rows as the chip's workgroups hold at a time, in each one's range and past it."""
    p = problem(T, H, rt, dt, gate="channel")
    p["R"][T // 2] *= 1e-18                       # (with this eps the sums of one row are in 64 bits)
    check_bwd(p, alpha=0.5, eps=1e-8)


@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("H", [768, 770, 9000])
def test_norm_bwd_parts(gate, post, pre, H):
    check_bwd(problem(21, H, F, B, True, post, gate, pre), alpha=-0.25)


def test_norm_bwd_without_a_block():
    for H in (64, 65, 9000):
        check_bwd(problem(30, H, F, B, block=False))
        check_bwd(problem(30, H, B, B, block=False), with_dR=False)


def test_norm_bwd_many_rows():
    check_bwd(problem(3000, 136, B, B, gate="channel"))
    check_bwd(problem(700, 4096, B, B, gate="token"))


def test_norm_bwd_no_rows():
    p = problem(0, 40, F, F, gate="channel")
    got = check_bwd(p)
    for name in ("dw_post", "dgate", "dw_pre"):
        assert getattr(got, name).shape == (40,) and not getattr(got, name).any()


def test_norm_bwd_far_sizes():
    for H in (64, 300, 9000):
        p = problem(8, H, F, F, gate="channel")
        p["R"][0], p["Y"][0] = 0, 0
        p["Y"][2] *= 1e30
        p["R"][3] *= 1e30
        p["Y"][4] *= 1e-30
        p["R"][5] *= 1e-30
        check_bwd(p)


def test_norm_bwd_zero_gate():
    """A gate of 0 has a gradient; the block behind it none."""
    p = problem(6, 100, F, F, gate="token")
    p["gate"][2] = 0
    got = check_bwd(p)
    assert not n(got.dY)[2].any() and n(got.dgate)[2, 0] != 0
    p = problem(6, 100, F, F, gate="channel")
    p["gate"][7] = 0
    got = check_bwd(p)
    assert n(got.dgate)[7] != 0 and n(got.dw_post)[7] == 0


def test_norm_bwd_against_differences():
    """Of the forward operator itself, in FP32, moved by 2 h along a direction: outputs
    within 48 u of values up to 4, so the quotient of the T H sum errs by at most 48 u 4 T H
    / (2 h) and, their third derivatives below 50, 10 h^2 T H."""
    T, H, h = 3, 64, 2.0 ** -7
    for gate in ("channel", "token"):
        p = problem(T, H, F, F, gate=gate, seed=5)
        p["Y"] /= 3
        g = torch.Generator().manual_seed(6)
        dR, dN = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)

        def f(q):
            o = dg.residual_norm(dev(q["R"]), dev(q["Y"]), w_post=dev(q["w_post"]), gate=dev(q["gate"]), alpha=0.5,
                                 w_pre=dev(q["w_pre"]), eps=1e-3)
            return float((o.R.double().cpu() * dR + o.N.double().cpu() * dN).sum())

        stream = dg.residual_norm(dev(p["R"]), dev(p["Y"]), w_post=dev(p["w_post"]), gate=dev(p["gate"]), alpha=0.5,
                                  w_pre=dev(p["w_pre"]), eps=1e-3).R
        got = dg.residual_norm_bwd(dev(dR), dev(dN), stream, dev(p["Y"]), w_post=dev(p["w_post"]), gate=dev(p["gate"]),
                                   alpha=0.5, w_pre=dev(p["w_pre"]), eps=1e-3)
        for name, key in (("dR", "R"), ("dY", "Y"), ("dw_post", "w_post"), ("dgate", "gate"), ("dw_pre", "w_pre")):
            d = torch.rand(p[key].shape, generator=g) * 2 - 1
            d /= d.norm()
            want = (f(dict(p, **{key: p[key] + h * d})) - f(dict(p, **{key: p[key] - h * d}))) / (2 * h)
            have = float((getattr(got, name).double().cpu() * d).sum())
            bound = 48 * U * 4 * T * H / (2 * h) + 10 * h * h * (T * H) ** 0.5
            assert abs(have - want) <= bound, (gate, name, have, want, bound)


# ---------------------------------------------------------------- calls

def test_norm_repeatable_and_on_a_side_stream():
    p = problem(2000, 1424, B, B, gate="channel")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for a, b in zip(check(p), check(p, stream=s)):
        assert (a is None and b is None) or torch.equal(a, b)
    for a, b in zip(check_bwd(p), check_bwd(p, stream=s)):
        assert torch.equal(a, b)


def test_norm_graph():
    p = {k: dev(v) for k, v in problem(300, 512, B, B, gate="token").items()}
    dN = torch.randn(300, 512, device=DEV).to(B)

    def step():
        o = dg.residual_norm(p["R"], p["Y"], w_post=p["w_post"], gate=p["gate"], w_pre=p["w_pre"], codes="pow2")
        return (*o, *dg.residual_norm_bwd(dN, dN, o.R, p["Y"], w_post=p["w_post"], gate=p["gate"], w_pre=p["w_pre"]))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        for k, v in problem(300, 512, B, B, gate="token", seed=seed).items():
            p[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_norm_refusals():
    x, w = torch.zeros(6, 32, device=DEV), torch.ones(32, device=DEV)
    for bad in (lambda: dg.residual_norm(x), lambda: dg.residual_norm(x, w_post=w, w_pre=w),
                lambda: dg.residual_norm(x, x[:5], w_pre=w), lambda: dg.residual_norm(x, w_pre=w[:31]),
                lambda: dg.residual_norm(x, x, gate=w[:6]), lambda: dg.residual_norm(x, x, gate=torch.ones(1, 6, device=DEV)),
                lambda: dg.residual_norm(x.t(), w_pre=w), lambda: dg.residual_norm(x, x, codes="pow2"),
                lambda: dg.residual_norm(x, x, w_pre=w, values=False), lambda: dg.residual_norm(x, x, dtype="bf16"),
                lambda: dg.residual_norm_bwd(None, None, x, x), lambda: dg.residual_norm_bwd(x, x, x, x),
                lambda: dg.residual_norm_bwd(x, None, x, w_pre=w), lambda: dg.residual_norm_bwd(x, None, None),
                lambda: dg.residual_norm_bwd(x, x, x, x.bfloat16(), w_pre=w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dg.residual_norm(x, w_pre=w.double()), lambda: dg.residual_norm(x.half(), w_pre=w),
                lambda: dg.residual_norm_bwd(x.bfloat16(), x, x, w_pre=w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dg.residual_norm(x, w_pre=w, eps=0.0), lambda: dg.residual_norm(x, x, alpha=float("nan")),
                lambda: dg.residual_norm(torch.zeros(2, 24, device=DEV), w_pre=w[:24].clone(), codes="pow2"),
                lambda: dg.residual_norm(x[:, :0].contiguous(), w_pre=w[:0])):
        with pytest.raises(dg.DGError):
            bad()
