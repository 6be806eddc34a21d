"""The measured cases of the MoE feed-forward operators around the FP8 products.

dispatch      tokens sorted by expert, their rows gathered and quantised
combine       expert outputs back to tokens, router weights applied
combine_bwd   its gradient: rows of dY and the gradient of the router weights
swiglu        the gated activation between the two products, which also keeps
              its input in 8 bits for the backward pass
swiglu_bwd    its gradient from that 8-bit checkpoint
wgrad         each expert's weight gradient from its 8-bit activations

`own` selects the framework's kernels; otherwise the operators are computed in
elementary torch operations.  8-bit results are float8 tensors beside their
scales.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # one token of a decode step: 2 of 64 experts, packed segments, codes for the next product
        dict(name="dispatch-one-token", op="dispatch", tokens=1, top_k=2, experts=64, hidden=2048, align=1,
             skew=1.0, drop=0.0, out="fp8", scale="amax", ids="i64"),
        # a large training batch over many experts, segments padded for the grouped product
        dict(name="dispatch-large", op="dispatch", tokens=16384, top_k=8, experts=256, hidden=4096, align=128,
             skew=0.5, drop=0.0, out="fp8", scale="pow2", ids="i32"),
        # the end of a decode step of 128 tokens
        dict(name="combine-decode", op="combine", tokens=128, top_k=2, experts=64, hidden=2048, align=1,
             skew=1.0, drop=0.0, dtype="bf16", weighted=True),
        # a training or prefill batch of the 64-expert layer, popular experts first
        dict(name="combine-train", op="combine", tokens=8192, top_k=2, experts=64, hidden=2048, align=128,
             skew=1.0, drop=0.0, dtype="bf16", weighted=True),
        # an odd token count, odd width, six choices each, a tenth of them dropped for lack of room
        dict(name="combine-bwd-odd", op="combine_bwd", tokens=1009, top_k=6, experts=60, hidden=1408, align=128,
             skew=1.0, drop=0.1, dtype="bf16"),
        # the backward pass of the 8-expert layer
        dict(name="combine-bwd-train", op="combine_bwd", tokens=4096, top_k=2, experts=8, hidden=4096, align=128,
             skew=0.0, drop=0.0, dtype="bf16"),
        # between the two products of a decode step
        dict(name="swiglu-decode", op="swiglu", rows=256, inner=2048),
        # between the two products of a training step
        dict(name="swiglu-train", op="swiglu", rows=9216, inner=4096),
        # a small microbatch, a width whose last scale block is partial
        dict(name="swiglu-bwd-odd", op="swiglu_bwd", rows=777, inner=1424),
        # the backward pass of the training step above
        dict(name="swiglu-bwd-train", op="swiglu_bwd", rows=9216, inner=4096),
        # weight gradient of the 8-expert layer into FP32
        dict(name="wgrad-8-experts", op="wgrad", tokens=4096, top_k=2, experts=8, n=4096, k=4096, skew=0.0,
             out="f32"),
        # weight gradient of the 64-expert layer, very uneven row counts, BF16 gradients
        dict(name="wgrad-64-experts", op="wgrad", tokens=8192, top_k=2, experts=64, n=2048, k=2048, skew=1.0,
             out="bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_bwd", "swiglu", "swiglu_bwd", "wgrad"])
    if op in ("swiglu", "swiglu_bwd"):
        return dict(op=op, rows=_log_int(rng, 1, 9000), inner=_log_int(rng, 256, 4096, 16))
    experts = _log_int(rng, 4, 256)
    top_k = rng.randint(1, min(8, experts))
    if op == "wgrad":
        experts = min(experts, 32)
        return dict(op=op, tokens=_log_int(rng, 16, 8192 // max(2, top_k)), top_k=min(top_k, experts),
                    experts=experts, n=_log_int(rng, 256, 2048, 16), k=_log_int(rng, 256, 2048, 16),
                    skew=rng.choice([0.0, 0.5, 1.0]), out=rng.choice(["f32", "bf16"]))
    c = dict(op=op, tokens=_log_int(rng, 1, 16384), top_k=top_k, experts=experts,
             hidden=_log_int(rng, 256, 4096, 16), align=rng.choice([1, 128]), skew=rng.choice([0.0, 0.5, 1.0]),
             drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "dispatch":
        c.update(out=rng.choice(["fp8", "fp8", "bf16"]), scale=rng.choice(["pow2", "amax"]),
                 ids=rng.choice(["i32", "i64"]))
    else:
        c.update(dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "combine":
            c.update(weighted=rng.choice([True, True, False]))
    return c


def _rows(c):
    """Rows of the sorted matrix: the most that the segments can take."""
    slots = c["tokens"] * c["top_k"]
    if c["align"] == 1:
        return slots
    return (slots + 127 * min(c["experts"], slots)) // 128 * 128


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ---------------------------------------------------------------- inputs

def _activations(g, rows, cols):
    """Rows of a residual stream: unit variance, a few columns far larger."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= 1 + 15 * (torch.rand(cols, generator=g, device="cuda") < 0.004)
    return x


def _route(g, c):
    """Each token's distinct experts and its router weights; expert popularity
    falls off as rank ** -skew.  A dropped choice has the id -1."""
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    logits = -c["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
    top = torch.topk(logits[torch.randperm(E, generator=g, device="cuda")] + noise, k, dim=1)
    ids = top.indices
    if c.get("drop", 0.0) > 0:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < c["drop"], -1, ids)
    return ids, torch.softmax(top.values, dim=1).contiguous()


def _sort_plain(ids, E, align, M):
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    count = torch.bincount(key, minlength=E + 1)
    seg = (count[:E] + align - 1) // align * align
    offs = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offs[1:] = torch.cumsum(seg, 0)
    order = torch.argsort(key, stable=True)
    sorted_key = key[order]
    first = torch.cumsum(count, 0) - count
    rank = torch.arange(T * k, device=ids.device) - first[sorted_key]
    row = torch.where(sorted_key < E, offs[sorted_key] + rank, M)      # M: a row past the end
    slot_row = torch.empty_like(row)
    slot_row[order] = row
    row_slot = torch.full((M + 1,), -1, dtype=torch.int32, device=ids.device)
    row_slot[slot_row] = torch.arange(T * k, dtype=torch.int32, device=ids.device)
    offs[E] = M
    slot_row = torch.where(slot_row < M, slot_row, -1)
    return (offs.to(torch.int32), count[:E].to(torch.int32), row_slot[:M].contiguous(),
            slot_row.to(torch.int32).reshape(T, k))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("swiglu", "swiglu_bwd"):
        h = _activations(g, c["rows"], 2 * c["inner"]).to(torch.bfloat16)
        h[torch.rand(c["rows"], generator=g, device="cuda") < 0.05] = 0          # padding rows
        if c["op"] == "swiglu":
            s["h"] = h
        else:
            I = c["inner"]
            q, sc = zip(*(_quantise(h[:, i * I:(i + 1) * I].float(), "pow2") for i in (0, 1)))
            s["hq"] = torch.cat(q, 1).to(torch.float8_e4m3fn).view(torch.uint8)
            s["sh"] = torch.stack(sc, 1).contiguous()
            s["da"] = torch.randn(c["rows"], I, generator=g, device="cuda").mul_(1e-2).to(torch.bfloat16)
        return s
    ids, w = _route(g, c)
    if c["op"] == "dispatch":
        s["ids"] = ids.to(torch.int32 if c["ids"] == "i32" else torch.int64).contiguous()
        s["x"] = _activations(g, c["tokens"], c["hidden"]).to(torch.bfloat16)
        return s
    M = _rows(dict(c, align=c.get("align", 128)))
    s["offs"], s["counts"], s["row_slot"], s["slot_row"] = _sort_plain(ids, c["experts"], c.get("align", 128), M)
    real = s["row_slot"] >= 0
    if c["op"] == "wgrad":
        x = _activations(g, M, c["k"]).to(torch.bfloat16) * real[:, None]
        q, s["sx"] = _quantise(x.float(), "pow2")
        s["x"] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        s["dy"] = torch.randn(M, c["n"], generator=g, device="cuda").mul_(1e-2).to(torch.bfloat16) * real[:, None]
        s["segments"] = list(zip(s["offs"].tolist(), s["counts"].tolist()))
        return s
    s["w"] = w
    s["y"] = (torch.randn(M, c["hidden"], generator=g, device="cuda") * real[:, None]).to(_dtype(c["dtype"]))
    if c["op"] == "combine_bwd":
        s["dout"] = torch.randn(c["tokens"], c["hidden"], generator=g, device="cuda").mul_(1e-2).to(
            _dtype(c["dtype"]))
    elif not c["weighted"]:
        s["w"] = None
    return s


# ---------------------------------------------------------------- plain forms

def _pow2(e):
    """2 ** e in 64 bits, exactly (|e| < 1022)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x, scale):
    """(values on the E4M3 grid, scales) of x, one scale for each row and 128
    columns; the quotients and their rounding in 64 bits."""
    rows, cols = x.shape
    kb = -(-cols // 128)
    xb = torch.nn.functional.pad(x, (0, 128 * kb - cols)).view(rows, kb, 128)
    amax = xb.abs().amax(2).double()
    if scale == "pow2":
        m, e = torch.frexp(amax / E4M3_MAX)
        s = _pow2(torch.where(m > 0.5, e, e - 1).clamp(min=-126))
    else:
        s = (amax / E4M3_MAX).float().double()
    s = torch.where(amax > 0, s, 1.0)
    v = xb.double() / s[:, :, None]
    step = _pow2(torch.frexp(v)[1].clamp(min=-5) - 4)
    q = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(rows, 128 * kb)[:, :cols].float(), s.float()


def _decode(q, s):
    """32-bit values of codes q with one scale for each row and 128 columns."""
    rows, cols = q.shape
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1)[:, :cols]


def _rows_of(values, index):
    """values[index], zeros where the index is negative."""
    return values[index.clamp(min=0)] * (index >= 0).unsqueeze(-1)


def _dispatch_plain(s):
    c = s["case"]
    offs, counts, row_slot, slot_row = _sort_plain(s["ids"], c["experts"], c["align"], _rows(c))
    src = torch.where(row_slot >= 0, torch.div(row_slot, c["top_k"], rounding_mode="floor"), -1).long()
    if c["out"] == "bf16":
        return offs, counts, row_slot, slot_row, _rows_of(s["x"], src)
    q, sc = _quantise(s["x"].float(), c["scale"])
    q = _rows_of(q, src).to(torch.float8_e4m3fn)
    return offs, counts, row_slot, slot_row, q, torch.where(src[:, None] >= 0, sc[src.clamp(min=0)], 1.0)


def _combine_plain(s):
    rows = _rows_of(s["y"].float(), s["slot_row"].long())
    if s["w"] is not None:
        rows = rows * s["w"].unsqueeze(-1)
    return rows.sum(1).to(s["y"].dtype)


def _combine_bwd_plain(s):
    k, slots, dout = s["case"]["top_k"], s["row_slot"].long(), s["dout"].float()
    w = s["w"].reshape(-1)
    token = torch.where(slots >= 0, torch.div(slots, k, rounding_mode="floor"), -1)
    dy = _rows_of(dout, token) * w[slots.clamp(min=0)].unsqueeze(-1)
    dw = (_rows_of(s["y"].float(), s["slot_row"].long()) * dout.unsqueeze(1)).sum(2)
    return dy.to(s["y"].dtype), dw


def _swiglu_plain(s):
    I = s["case"]["inner"]
    h = s["h"].float()
    g, u = h[:, :I].double(), h[:, I:].double()
    # in 64 bits: the rounding to 8 bits turns on values next to a border
    qa, sa = _quantise(u * g / (1 + torch.exp(-g)), "pow2")
    qg, sg = _quantise(h[:, :I], "pow2")
    qu, su = _quantise(h[:, I:], "pow2")
    return (qa.to(torch.float8_e4m3fn), sa, torch.cat([qg, qu], 1).to(torch.float8_e4m3fn),
            torch.stack([sg, su], 1))


def _swiglu_bwd_plain(s):
    I = s["case"]["inner"]
    g, u = _decode(s["hq"][:, :I], s["sh"][:, 0]), _decode(s["hq"][:, I:], s["sh"][:, 1])
    da, sig = s["da"].float(), 1 / (1 + torch.exp(-g))
    return torch.cat([da * u * sig * (1 + g * (1 - sig)), da * g * sig], 1).to(torch.bfloat16)


def _wgrad_plain(s):
    x, dy = _decode(s["x"], s["sx"]), s["dy"].float()
    dw = torch.stack([dy[o:o + n].t() @ x[o:o + n] for o, n in s["segments"]])
    return dw.to(_dtype(s["case"]["out"]))


_PLAIN = {"dispatch": _dispatch_plain, "combine": _combine_plain, "combine_bwd": _combine_bwd_plain,
          "swiglu": _swiglu_plain, "swiglu_bwd": _swiglu_bwd_plain, "wgrad": _wgrad_plain}


# ---------------------------------------------------------------- the framework's operators

def _dispatch_own(s):
    from moe_grouped_gemm_block_amd import dg
    c = s["case"]
    plan = dg.moe_sort(s["ids"], c["experts"], align=c["align"])
    if c["out"] == "bf16":
        return (*plan, dg.moe_permute(s["x"], plan.slot_row, plan.row_slot))
    q, sc = dg.moe_permute_fp8(s["x"], plan.slot_row, plan.row_slot, scale=c["scale"])
    return (*plan, q.view(torch.float8_e4m3fn), sc)


def _combine_own(s):
    from moe_grouped_gemm_block_amd import dg
    return dg.moe_combine(s["y"], s["slot_row"], s["w"])


def _combine_bwd_own(s):
    from moe_grouped_gemm_block_amd import dg
    return dg.moe_combine_bwd(s["dout"], s["y"], s["slot_row"], s["row_slot"], s["w"])


def _swiglu_own(s):
    from moe_grouped_gemm_block_amd import dg
    a, sa, hq, sh = dg.swiglu_fp8(s["h"])
    return a.view(torch.float8_e4m3fn), sa, hq.view(torch.float8_e4m3fn), sh


def _swiglu_bwd_own(s):
    from moe_grouped_gemm_block_amd import dg
    return dg.swiglu_fp8_bwd(s["da"], s["hq"], s["sh"])


def _wgrad_own(s):
    from moe_grouped_gemm_block_amd import dg
    return dg.grouped_wgrad_fp8(s["dy"], s["x"], s["sx"], s["offs"], s["counts"], out_dtype=s["case"]["out"])


_OWN = {"dispatch": _dispatch_own, "combine": _combine_own, "combine_bwd": _combine_bwd_own,
        "swiglu": _swiglu_own, "swiglu_bwd": _swiglu_bwd_own, "wgrad": _wgrad_own}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] in ("swiglu", "swiglu_bwd"):
        M, I, kb = c["rows"], c["inner"], -(-c["inner"] // 128)
        if c["op"] == "swiglu":          # h in; codes of a and h and their scales out
            return {"bytes": M * (4 * I + 3 * I + 12 * kb), "flops": 8 * M * I}
        return {"bytes": M * (2 * I + 8 * kb + 2 * I + 4 * I), "flops": 16 * M * I}
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    slots = round(T * k * (1 - c.get("drop", 0.0)))
    if c["op"] == "wgrad":
        N, K = c["n"], c["k"]
        return {"bytes": slots * (2 * N + K + 4 * -(-K // 128)) + 4 * (2 * E + 1)
                + E * N * K * (4 if c["out"] == "f32" else 2), "flops": 2 * slots * N * K}
    H, M = c["hidden"], _rows(c)
    if c["op"] == "dispatch":
        row = 2 * H if c["out"] == "bf16" else H + 4 * -(-H // 128)
        return {"bytes": T * k * (8 if c["ids"] == "i64" else 4) + 4 * (2 * E + 1 + M + T * k) + 2 * T * H + M * row,
                "flops": 4 * T * H if c["out"] == "fp8" else 0}
    b = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "combine":
        return {"bytes": T * k * (8 if c["weighted"] else 4) + slots * H * b + T * H * b, "flops": 2 * slots * H}
    return {"bytes": T * k * 12 + 4 * M + T * H * b + slots * H * b + M * H * b, "flops": 3 * slots * H}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_codes(x, pow2):
    """Nearest of the 127 E4M3 magnitudes (ties to the even code) by search among
    their midpoints, for x in 64 bits; one scale for each row and 128 columns."""
    grid = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                         for c in range(127)], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    powers = torch.tensor([2.0 ** e for e in range(-126, 128)], dtype=torch.float64, device=x.device)
    values, scales = torch.empty_like(x), []
    for b in range(0, x.shape[1], 128):
        block = x[:, b:b + 128]
        amax = block.abs().max(dim=1, keepdim=True).values
        if pow2:
            s = powers[torch.searchsorted(448 * powers, amax, right=False)]     # the least that holds amax
        else:
            s = (amax / 448).to(torch.float32).to(torch.float64)
        s = torch.where(amax == 0, torch.ones_like(s), s)
        v = (block / s).abs().contiguous()
        lo = torch.searchsorted(mid, v, right=False)          # midpoints below v
        tie = (lo < 126) & (mid[lo.clamp(max=125)] == v) & (lo % 2 == 1)
        values[:, b:b + 128] = torch.copysign(grid[lo + tie.long()], block)
        scales.append(s)
    return values, torch.cat(scales, 1)


def exact(case, seed):
    c = case
    if c["op"] == "dispatch" and c["out"] == "bf16":
        return None                                           # copies and whole numbers only
    s = prepare(case, seed)
    if c["op"] == "dispatch":
        q, sc = _exact_codes(s["x"].double(), c["scale"] == "pow2")
        ids = s["ids"].cpu().reshape(-1).tolist()
        E, k, M = c["experts"], c["top_k"], _rows(c)
        slots = [[] for _ in range(E)]
        for slot, e in enumerate(ids):
            if 0 <= e < E:
                slots[e].append(slot)
        rows = []
        for group in slots:
            rows += group + [-1] * (-len(group) % c["align"])
        rows = torch.tensor(rows + [-1] * (M - len(rows)), device="cuda")
        codes = torch.zeros(M, c["hidden"], dtype=torch.float64, device="cuda")
        scales = torch.ones(M, q.shape[1] // 128 + (q.shape[1] % 128 > 0), dtype=torch.float64, device="cuda")
        at = torch.nonzero(rows >= 0).flatten()
        codes[at], scales[at] = q[rows[at] // k], sc[rows[at] // k]
        return None, None, None, None, codes, scales
    if c["op"] == "swiglu":
        g, u = s["h"].double().split(c["inner"], dim=1)
        a, sa = _exact_codes(u * (g * torch.sigmoid(g)), True)
        qg, sg = _exact_codes(g.contiguous(), True)
        qu, su = _exact_codes(u.contiguous(), True)
        return a, sa, torch.cat([qg, qu], 1), torch.stack([sg, su], 1)
    if c["op"] == "swiglu_bwd":
        I = c["inner"]
        col = torch.arange(I, device="cuda") // 128
        h = s["hq"].view(torch.float8_e4m3fn).double()
        g = h[:, :I] * s["sh"][:, 0][:, col]
        u = h[:, I:] * s["sh"][:, 1][:, col]
        p = torch.sigmoid(g)
        da = s["da"].double()
        return torch.cat([da * u * (p + g * p * (1 - p)), da * (g * p)], 1)
    if c["op"] == "wgrad":
        x = s["x"].view(torch.float8_e4m3fn).double() * s["sx"][:, torch.arange(c["k"], device="cuda") // 128]
        dw = torch.zeros(c["experts"], c["n"], c["k"], dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            o, n = int(s["offs"][e]), int(s["counts"][e])
            dw[e] = torch.matmul(s["dy"][o:o + n].double().t().contiguous(), x[o:o + n])
        return dw
    T, k, H = c["tokens"], c["top_k"], c["hidden"]
    if c["op"] == "combine":
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            here = torch.nonzero(s["slot_row"][:, j] >= 0).flatten()
            rows = s["y"][s["slot_row"][here, j].long()].double()
            out[here] += rows if s["w"] is None else rows * s["w"][here, j:j + 1].double()
        return out
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        here = torch.nonzero(s["slot_row"][:, j] >= 0).flatten()
        at = s["slot_row"][here, j].long()
        d = s["dout"][here].double()
        dy[at] = d * s["w"][here, j:j + 1].double()
        dw[here, j] = (d * s["y"][at].double()).sum(1)
    return dy, dw
