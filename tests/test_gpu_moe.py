"""Tokens sorted by expert and back, and the gradients, against the float64 /
integer oracle.  Needs a GPU.

Tolerances.  A BF16 result is off by at most half a step, 2^-8 of the value, an
FP32 one by 2^-24; before that rounding an FP32 sum of n products taken with
fused multiply-adds is off by at most n 2^-24 of the sum of magnitudes (first
order), and the dot products add one rounding per lane step of their reduction."""
import sys

import numpy as np
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from oracle import moe as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


def make_ids(T, k, G, seed, kind="random", drop=0.0):
    rng = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full((T, k), G - 1)
    elif kind == "none":
        ids = np.full((T, k), -1)
    elif kind == "skew":
        ids = np.minimum(rng.geometric(0.3, (T, k)) - 1, G - 1)
    else:
        ids = rng.integers(0, G, (T, k))
    if drop:
        ids = np.where(rng.random((T, k)) < drop, rng.choice([-1, -5, G, G + 1000], (T, k)), ids)
    return ids


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def plan_for(T, k, G, align, seed, **kw):
    ids = make_ids(T, k, G, seed, **kw)
    M = O.rows_needed(T, k, G, align)
    ref = O.sort(ids, G, align, M)
    return ids, M, ref, dg.moe_sort(dev(ids.astype(np.int32)), G, align=align)


@pytest.mark.parametrize("align", [1, 128])
@pytest.mark.parametrize("T,k,G,kind,drop,it", [
    (0, 2, 5, "random", 0, np.int32), (1, 1, 1, "random", 0, np.int32), (1, 2, 64, "random", 0, np.int64),
    (3, 8, 8, "random", 0.3, np.int32), (127, 2, 3, "one", 0, np.int32), (130, 3, 7, "none", 0, np.int64),
    (500, 4, 1000, "random", 0.1, np.int32), (1000, 8, 1024, "skew", 0, np.int64),
    (1024, 8, 64, "skew", 0, np.int32), (1025, 8, 64, "random", 0.5, np.int64),
    (4099, 3, 257, "skew", 0.05, np.int32), (20011, 8, 256, "random", 0, np.int64),
    (40000, 7, 1024, "one", 0, np.int32)])
def test_sort(T, k, G, kind, drop, it, align):
    log(f"sort T={T} k={k} G={G} {kind} drop={drop} align={align}")
    ids = make_ids(T, k, G, seed=T + k, kind=kind, drop=drop).astype(it)
    for extra in (0, 2 * align):
        M = O.rows_needed(T, k, G, align) + extra
        plan = dg.moe_sort(dev(ids), G, align=align, rows=M)
        torch.cuda.synchronize()
        for name, got, want in zip(plan._fields, plan, O.sort(ids, G, align, M)):
            assert np.array_equal(got.cpu().numpy(), want), name


def test_sort_ids_beyond_32_bits():
    """64-bit ids whose low halves look like experts are dropped."""
    ids = np.array([[(1 << 32) + 1, 1], [-(1 << 40), 0]])
    plan = dg.moe_sort(dev(ids), 4, align=1)
    for got, want in zip(plan, O.sort(ids, 4, 1, 4)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_refuses_too_few_rows():
    with pytest.raises(dg.DGError):
        dg.moe_sort(torch.zeros(10, 2, dtype=torch.int32, device=DEV), 4, align=128, rows=128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,G,H,align,drop", [
    (1, 2, 64, 2048, 1, 0), (5, 1, 2, 1, 128, 0), (70, 3, 4, 7, 1, 0.4), (33, 8, 16, 200, 128, 0.2),
    (129, 2, 8, 1000, 128, 0), (64, 6, 60, 1408, 1, 1.0)])
def test_permute(T, k, G, H, align, drop, dtype):
    log(f"permute T={T} k={k} G={G} H={H} align={align} drop={drop} {dtype}")
    _, M, ref, plan = plan_for(T, k, G, align, seed=T, drop=drop)
    x = dev(np.random.default_rng(H).standard_normal((T, H)), DTYPE[dtype])
    Y = torch.full((M, H), float("nan"), dtype=DTYPE[dtype], device=DEV)
    got = dg.moe_permute(x, plan.slot_row, plan.row_slot, Y=Y)
    torch.cuda.synchronize()
    assert np.array_equal(got.float().cpu().numpy(), O.permute(x.float().cpu().numpy(), ref[2], k))


def awkward_values(T, H, rng):
    """Rows of very different size, zero blocks, subnormals, block maxima at and
    next to 448 times a power of two, and values half way between codes."""
    x = (rng.standard_normal((T, H)) * np.exp2(rng.uniform(-30, 30, (T, 1)))).astype(np.float32)
    for t in range(T):
        if t % 7 == 1:
            x[t] = 0
        elif t % 7 == 2:
            x[t, :min(H, 128)] = 0
        elif t % 7 == 3:
            x[t] = (x[t] / np.abs(x[t]).max() * np.float32(1e-38)).astype(np.float32)
        elif t % 7 == 4:
            x[t] = np.round(rng.uniform(-448, 448, H)).astype(np.float32)
            x[t, ::128] = 448
        elif t % 7 == 5:
            x[t] = rng.choice([0.5, 1.0, 17.0, 19.0, 2.0 ** -7, 3 * 2.0 ** -10], H).astype(np.float32)
            x[t, ::128] = np.nextafter(np.float32(448), np.float32(500)) if t % 2 else np.float32(224)
    return x


@pytest.mark.parametrize("scale", ["pow2", "amax"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,G,H,align,drop", [
    (1, 2, 64, 2048, 1, 0), (9, 1, 2, 16, 128, 0), (70, 3, 4, 144, 1, 0.4), (130, 2, 8, 1424, 128, 0.1),
    (64, 6, 60, 512, 128, 1.0)])
def test_permute_fp8(T, k, G, H, align, drop, dtype, scale):
    log(f"permute_fp8 T={T} k={k} G={G} H={H} align={align} drop={drop} {dtype} {scale}")
    _, M, ref, plan = plan_for(T, k, G, align, seed=T, drop=drop)
    x = dev(awkward_values(T, H, np.random.default_rng(H + T)), DTYPE[dtype])
    Q = torch.full((M, H), 0xFF, dtype=torch.uint8, device=DEV)
    S = torch.full((M, -(-H // 128)), float("nan"), device=DEV)
    dg.moe_permute_fp8(x, plan.slot_row, plan.row_slot, scale=scale, Q=Q, S=S)
    torch.cuda.synchronize()
    q, s = O.quantise(x.double().cpu().numpy(), scale == "pow2")
    assert np.array_equal(S.cpu().numpy(), O.permute(s, ref[2], k, fill=1))
    assert np.array_equal(Q.cpu().numpy(), O.permute(q, ref[2], k))


COMBINE_SHAPES = [(1, 2, 64, 2048, 1, 0), (5, 1, 2, 1, 128, 0), (70, 3, 4, 9, 1, 0.4), (33, 8, 16, 200, 128, 0.2),
                  (129, 5, 8, 1004, 128, 0), (12, 11, 16, 72, 1, 0.1), (40, 6, 60, 1408, 1, 1.0)]


def layer_data(T, k, G, H, align, drop, dtype, seed):
    """A plan, Y with NaN in rows of padding, weights with NaN at dropped choices."""
    _, M, ref, plan = plan_for(T, k, G, align, seed=seed, drop=drop)
    rng = np.random.default_rng(seed + 1)
    y = dev(rng.standard_normal((M, H)), DTYPE[dtype])
    y[dev(ref[2] < 0)] = float("nan")
    w = rng.random((T, k)).astype(np.float32)
    w[ref[3] < 0] = np.nan
    return M, ref, plan, y, w, rng


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,G,H,align,drop", COMBINE_SHAPES)
def test_combine(T, k, G, H, align, drop, dtype, weighted):
    log(f"combine T={T} k={k} G={G} H={H} align={align} drop={drop} {dtype} weighted={weighted}")
    M, ref, plan, y, w, _ = layer_data(T, k, G, H, align, drop, dtype, seed=H + T)
    out = torch.full((T, H), float("nan"), dtype=DTYPE[dtype], device=DEV)
    dg.moe_combine(y, plan.slot_row, dev(w) if weighted else None, out=out)
    torch.cuda.synchronize()
    want, mass = O.combine(y.float().cpu().numpy(), ref[3], w if weighted else None)
    err = np.abs(out.double().cpu().numpy() - want)
    before = k * 2.0 ** -24 * mass
    bound = before + HALF_STEP[dtype] * (np.abs(want) + before)
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,G,H,align,drop", COMBINE_SHAPES)
def test_combine_bwd(T, k, G, H, align, drop, dtype):
    log(f"combine_bwd T={T} k={k} G={G} H={H} align={align} drop={drop} {dtype}")
    M, ref, plan, y, w, rng = layer_data(T, k, G, H, align, drop, dtype, seed=H + T + 5)
    d = dev(rng.standard_normal((T, H)), DTYPE[dtype])
    dY = torch.full((M, H), float("nan"), dtype=DTYPE[dtype], device=DEV)
    dw = torch.full((T, k), float("nan"), device=DEV)
    dg.moe_combine_bwd(d, y, plan.slot_row, plan.row_slot, dev(w), dY=dY, dweights=dw)
    torch.cuda.synchronize()
    dy_o, dw_o, mass = O.combine_bwd(d.float().cpu().numpy(), y.float().cpu().numpy(), ref[3], w)
    err = np.abs(dY.double().cpu().numpy() - dy_o)
    # the product in FP32, then the output type
    assert np.all(err <= np.abs(dy_o) * (2.0 ** -24 + HALF_STEP[dtype] * (1 + 2.0 ** -24)))
    # a lane adds at most ceil(H / 64) + 8 products, the reduction 10 more sums
    n = -(-H // 64) + 8 + 10
    assert np.all(np.abs(dw.double().cpu().numpy() - dw_o) <= n * 2.0 ** -24 * mass)


def test_permute_and_combine_are_adjoint():
    """<permute(x), y> = <x, combine(y)> on whole numbers, where every sum is exact."""
    _, M, _, plan = plan_for(300, 4, 16, 128, seed=3, drop=0.2)
    rng = np.random.default_rng(4)
    x, y = (dev(rng.integers(-8, 9, (n, 264)), torch.float32) for n in (300, M))
    px = dg.moe_permute(x, plan.slot_row, plan.row_slot)
    cy = dg.moe_combine(y, plan.slot_row)
    assert float((px.double() * y.double()).sum()) == float((x.double() * cy.double()).sum())


def test_rows_past_32_bit_offsets():
    """Rows of Y and X whose byte offsets pass 2^32: a sampled token's rows."""
    T, k, G, H = 40000, 2, 4, 32768
    ids = make_ids(T, k, G, seed=9)
    plan = dg.moe_sort(dev(ids.astype(np.int32)), G, align=128)
    x = torch.randn(T, H, device=DEV, dtype=torch.bfloat16)
    y = dg.moe_permute(x, plan.slot_row, plan.row_slot)
    q, s = dg.moe_permute_fp8(x, plan.slot_row, plan.row_slot)
    out = dg.moe_combine(y, plan.slot_row)
    ones = torch.ones(T, k, device=DEV)
    dy, dw = dg.moe_combine_bwd(x, y, plan.slot_row, plan.row_slot, ones)
    at = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV)
    rows = plan.slot_row[at].long()
    assert int(rows.max()) * H * 2 > 1 << 32
    assert torch.equal(y[rows], x[at][:, None].expand(-1, k, -1))
    assert torch.equal(out[at], (x[at].float() * 2).bfloat16())
    assert torch.equal(dy[rows], y[rows])
    want = (x[at].double() ** 2).sum(1)
    assert torch.allclose(dw[at].double(), want[:, None].expand(-1, k), rtol=(H // 64 + 18) * 2.0 ** -24, atol=0)
    codes, scales = O.quantise(x[at].double().cpu().numpy(), True)
    assert np.array_equal(q[rows[:, 1]].cpu().numpy(), codes) and np.array_equal(s[rows[:, 1]].cpu().numpy(), scales)


def test_grids_past_32_bit_work_items():
    """A thread per element of an odd width, a workgroup per token, eight threads
    per block: more work-items than one dimension of a grid has (2^32, or the 2^31
    from which workgroups are laid out in two)."""
    T, H = 1048577, 4099
    assert T * H > 1 << 32
    y = torch.randn(5, H, device=DEV).bfloat16()
    slot = (torch.arange(T, device=DEV, dtype=torch.int32) % 5)[:, None].contiguous()
    out = dg.moe_combine(y, slot)
    for t in range(0, T, 1 << 17):
        assert torch.equal(out[t:t + (1 << 17)], y[slot[t:t + (1 << 17), 0].long()])
    at = [0, 1, (1 << 31) // H + 1, T - 2, T - 1]
    slot.fill_(-1)
    slot[at, 0] = torch.tensor([4, 0, 3, 1, 6], device=DEV, dtype=torch.int32)
    row_slot = torch.tensor([at[1], at[3], -1, at[2], at[0], -1, at[4]], device=DEV, dtype=torch.int32)
    got = dg.moe_permute(out, slot, row_slot)
    for r, t in enumerate(row_slot.tolist()):
        assert torch.equal(got[r], out[t]) if t >= 0 else not got[r].any()
    del out, got

    T, H = (1 << 24) + 3, 8
    at = [0, 1 << 23, T - 1]
    d = torch.randn(T, H, device=DEV)
    y = torch.randn(4, H, device=DEV)
    slot = torch.full((T, 1), -1, device=DEV, dtype=torch.int32)
    slot[at, 0] = torch.tensor([2, 0, 1], device=DEV, dtype=torch.int32)
    row_slot = torch.tensor([at[1], at[2], at[0], -1], device=DEV, dtype=torch.int32)
    dy, dw = dg.moe_combine_bwd(d, y, slot, row_slot, torch.ones(T, 1, device=DEV))
    assert torch.equal(dy[:3], d[row_slot[:3].long()]) and not dy[3].any()
    assert torch.count_nonzero(dw) == 3
    want = (d[at].double() * y[slot[at, 0].long()].double())
    assert bool(((dw[at, 0].double() - want.sum(1)).abs() <= 18 * 2.0 ** -24 * want.abs().sum(1)).all())
    del d, dw

    T, H = (1 << 28) + 3, 16
    at = [0, 1 << 27, T - 1]
    x = torch.zeros(T, H, device=DEV, dtype=torch.bfloat16)
    x[at] = torch.randn(3, H, device=DEV).bfloat16()
    slot = torch.full((T, 1), -1, device=DEV, dtype=torch.int32)
    slot[at, 0] = torch.arange(3, device=DEV, dtype=torch.int32)
    row_slot = torch.tensor(at + [-1], device=DEV, dtype=torch.int32)
    q, s = dg.moe_permute_fp8(x, slot, row_slot)
    codes, scales = O.quantise(x[at].double().cpu().numpy(), True)
    assert np.array_equal(q[:3].cpu().numpy(), codes) and np.array_equal(s[:3].cpu().numpy(), scales)
    assert not q[3].any() and float(s[3]) == 1
    del slot
    h = x.new_zeros(T, 2 * H)
    h[at] = torch.randn(3, 2 * H, device=DEV).bfloat16()
    for got, want in zip(dg.swiglu_fp8(h), dg.swiglu_fp8(h[at])):
        assert torch.equal(got[at], want)


def test_plan_of_most_rows():
    """As many rows as are counted in 32 bits: the rest of them is padding."""
    M = (1 << 31) - 1
    for T in (3, 4097):                                          # one workgroup, several
        ids = make_ids(T, 2, 4, seed=3)
        plan = dg.moe_sort(dev(ids.astype(np.int32)), 4, align=1, rows=M)
        short = dg.moe_sort(dev(ids.astype(np.int32)), 4, align=1)
        n = short.row_slot.numel()
        assert torch.equal(plan.slot_row, short.slot_row) and torch.equal(plan.row_slot[:n], short.row_slot)
        assert int(plan.row_slot[n:].max()) == -1 and int(plan.row_slot[n:].min()) == -1
        assert int(plan.group_offsets[-1]) == M
        del plan


def test_another_stream_and_poisoned_memory():
    """Calls on a stream of their own, with inputs written there just before."""
    _, M, ref, _ = plan_for(257, 4, 16, 128, seed=1)
    ids = make_ids(257, 4, 16, 1)
    side = torch.cuda.Stream()
    x = torch.randn(257, 512, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        xs = (x * 2).bfloat16()
        i32 = dev(ids.astype(np.int32))
    plan = dg.moe_sort(i32, 16, stream=side)
    y = dg.moe_permute(xs, plan.slot_row, plan.row_slot, stream=side)
    out = dg.moe_combine(y, plan.slot_row, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, (xs.float() * 4).bfloat16())
    assert np.array_equal(plan.row_slot.cpu().numpy(), ref[2])


def test_wrong_plans_are_refused():
    plan = dg.moe_sort(torch.zeros(10, 2, dtype=torch.int32, device=DEV), 4, align=1)
    x = torch.zeros(10, 64, device=DEV)
    with pytest.raises(ValueError):
        dg.moe_permute(x[:9], plan.slot_row, plan.row_slot)
    with pytest.raises(ValueError):
        dg.moe_permute(x.t(), plan.slot_row, plan.row_slot)
    with pytest.raises(TypeError):
        dg.moe_permute(x, plan.slot_row.long(), plan.row_slot)
    with pytest.raises(ValueError):
        dg.moe_combine(x, plan.slot_row, torch.ones(10, 3, device=DEV))
    with pytest.raises(dg.DGError):
        dg.moe_permute_fp8(torch.zeros(10, 40, device=DEV), plan.slot_row, plan.row_slot)
