"""The measured cases of the operators that make the MoE layer a block of a model.

route      each token's experts and their weights from the router's logits, with
           per-expert counts and the balance loss
route_bwd  the gradient of the logits from those of the weights and of the loss
norm       the residual stream past a block: the block's output normalised, gated,
           scaled and added, and the sum normalised for the next block, as values
           or as 8-bit codes with their scales
norm_bwd   its gradient, weights and gates included
clip       the global norm of many gradients, and their clipping

`own` selects the framework's kernels; otherwise the operators are computed in
elementary torch operations.  8-bit results are float8 tensors beside their
scales.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one token of a decode step: 2 of 64 experts
        dict(name="route-one-token", op="route", tokens=1, experts=64, top_k=2, score="softmax", renorm=True, scale=1.0,
             bias=False, dtype="f32", masked=0.0, closed=0.0, balance=False),
        # a training batch of the 64-expert layer
        dict(name="route-64-experts", op="route", tokens=8192, experts=64, top_k=2, score="softmax", renorm=True,
             scale=1.0, bias=False, dtype="bf16", masked=0.0, closed=0.0, balance=True),
        # a large training batch over many experts, their load evened out by a bias that only the choice sees
        dict(name="route-256-experts", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid", renorm=True,
             scale=2.5, bias=True, dtype="f32", masked=0.0, closed=0.0, balance=True),
        # an odd padded batch, six choices each, a third of the experts closed to a token
        dict(name="route-bwd-odd", op="route_bwd", tokens=1009, experts=60, top_k=6, score="softmax", renorm=False,
             scale=1.0, dtype="bf16", masked=0.1, closed=0.3, balance=True),
        # the backward pass of the large batch
        dict(name="route-bwd-256-experts", op="route_bwd", tokens=16384, experts=256, top_k=8, score="sigmoid",
             renorm=True, scale=2.5, dtype="f32", masked=0.0, closed=0.0, balance=True),
        # the first norm of a decode step of one token, straight to the product's codes
        dict(name="norm-one-token", op="norm", tokens=1, hidden=2048, block=False, post=False, gate="none", alpha=1.0,
             pre=True, out="codes", scale="pow2", stream="bf16", dtype="bf16"),
        # a microbatch of odd size, the stream in FP32, the block's output gated by channel
        dict(name="norm-odd", op="norm", tokens=777, hidden=1424, block=True, post=True, gate="channel", alpha=1.0,
             pre=True, out="both", scale="amax", stream="f32", dtype="bf16"),
        # between two blocks of a training step
        dict(name="norm-train", op="norm", tokens=8192, hidden=4096, block=True, post=True, gate="none", alpha=0.5,
             pre=True, out="values", scale="pow2", stream="bf16", dtype="bf16"),
        # an odd token count and width, a gate for each token, the stream in FP32
        dict(name="norm-bwd-odd", op="norm_bwd", tokens=1009, hidden=1408, block=True, post=True, gate="token",
             alpha=1.0, pre=True, stream="f32", dtype="bf16"),
        # the backward pass between two blocks of a training step, channels gated
        dict(name="norm-bwd-train", op="norm_bwd", tokens=8192, hidden=4096, block=True, post=True, gate="channel",
             alpha=0.5, pre=True, stream="bf16", dtype="bf16"),
        # the small parameters of a block: norms, gates, a router
        dict(name="clip-small", op="clip", layers=1, experts=8, hidden=257, inner=0, dtype="f32", out="f32",
             max_norm=1.0, size=1e-2),
        # the gradients of eight layers of 8 experts in BF16, clipped into FP32
        dict(name="clip-eight-layers", op="clip", layers=8, experts=8, hidden=1024, inner=1024, dtype="bf16",
             out="f32", max_norm=1.0, size=1e-2),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "norm", "norm_bwd", "clip"])
    if op in ("route", "route_bwd"):
        experts = _log_int(rng, 4, 256)
        c = dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, top_k=rng.randint(1, min(8, experts)),
                 score=rng.choice(["softmax", "sigmoid"]), renorm=rng.choice([True, True, False]),
                 scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.1]),
                 closed=rng.choice([0.0, 0.0, 0.3, 0.9]), balance=rng.choice([True, True, False]))
        if op == "route":
            c.update(bias=rng.choice([False, True]))
        return c
    if op == "clip":
        return dict(op=op, layers=rng.randint(1, 6), experts=rng.randint(2, 8), hidden=_log_int(rng, 64, 1024),
                    inner=rng.choice([0, _log_int(rng, 64, 1024)]), dtype=rng.choice(["f32", "bf16"]),
                    out=rng.choice(["f32", "same"]), max_norm=rng.choice([1.0, 1.0, 1e6]), size=rng.choice([1e-2, 10.0]))
    block = rng.choice([True, True, True, False])
    pre = not block or rng.choice([True, True, True, False])
    c = dict(op=op, tokens=_log_int(rng, 1, 8192), hidden=_log_int(rng, 256, 4096, rng.choice([16, 16, 16, 1])),
             block=block, post=block and rng.choice([True, True, False]),
             gate=rng.choice(["none", "channel", "token"]) if block else "none",
             alpha=rng.choice([1.0, 0.5]) if block else 1.0, pre=pre, stream=rng.choice(["bf16", "f32"]),
             dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        codes = pre and c["hidden"] % 16 == 0
        c.update(out=rng.choice(["values", "codes", "both"]) if codes else "values",
                 scale=rng.choice(["pow2", "amax"]))
    return c


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ---------------------------------------------------------------- inputs

def _logits(g, c):
    """The router's logits and the rows that hold a token.  Some experts are far
    more popular; a closed expert's logit is -inf, rows of padding hold anything."""
    T, E = c["tokens"], c["experts"]
    x = torch.randn(T, E, generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda")
    if c["closed"] > 0:
        x = torch.where(torch.rand(T, E, generator=g, device="cuda") < c["closed"], -math.inf, x)
    mask = None
    if c["masked"] > 0:
        mask = torch.rand(T, generator=g, device="cuda") >= c["masked"]
    return x.to(_dtype(c["dtype"])), mask


def _stream(g, rows, cols):
    """Rows of a residual stream: a few columns far larger than the others."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= 1 + 15 * (torch.rand(cols, generator=g, device="cuda") < 0.004)
    return x


def _shapes(c):
    """The parameters of `layers` layers: two norms, a gate, a router and, with an
    inner size, the experts' weights."""
    E, H, I = c["experts"], c["hidden"], c["inner"]
    layer = [(H,), (H,), (H,), (E, H)] + ([(E, 2 * I, H), (E, H, I)] if I else [])
    return layer * c["layers"]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("route", "route_bwd"):
        s["logits"], s["mask"] = _logits(g, c)
        E = c["experts"]
        if c["op"] == "route":
            s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if c["bias"] else None
            return s
        ids, _, counts, _, routed, _ = _route_plain(dict(s, bias=None))
        s["ids"], s["counts"], s["routed"] = ids, counts, routed
        s["dweights"] = torch.randn(ids.shape, generator=g, device="cuda") * 1e-2
        s["dloss"] = torch.full((), 0.01, device="cuda") if c["balance"] else None
        return s
    if c["op"] == "clip":
        s["grads"] = [(torch.randn(shape, generator=g, device="cuda") * c["size"]).to(_dtype(c["dtype"]))
                      for shape in _shapes(c)]
        s["out"] = [torch.empty_like(t, dtype=torch.float32 if c["out"] == "f32" else t.dtype) for t in s["grads"]]
        return s
    T, H = c["tokens"], c["hidden"]
    s["r"] = _stream(g, T, H).to(_dtype(c["stream"]))
    s["y"] = _stream(g, T, H).to(_dtype(c["dtype"])) if c["block"] else None
    for name, there in (("w_post", c["post"]), ("w_pre", c["pre"])):
        s[name] = 1 + 0.1 * torch.randn(H, generator=g, device="cuda") if there else None
    s["gate"] = None
    if c["gate"] == "channel":
        s["gate"] = torch.randn(H, generator=g, device="cuda") * 0.5
    elif c["gate"] == "token":
        s["gate"] = torch.rand(T, 1, generator=g, device="cuda")
    if c["op"] == "norm_bwd":
        s["dr"] = (torch.randn(T, H, generator=g, device="cuda") * 1e-2).to(_dtype(c["stream"]))
        s["dn"] = (torch.randn(T, H, generator=g, device="cuda") * 1e-2).to(_dtype(c["dtype"])) if c["pre"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _scores(x, score):
    """Scores and each token's probabilities of logits x; zeros in a row without an
    open expert."""
    if score == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
        return p, p
    s = 1 / (1 + torch.exp(-x))
    return s, s / s.sum(1, keepdim=True).clamp(min=1e-30)


def _route_plain(s):
    c = s["case"]
    x, k, E = s["logits"].float(), c["top_k"], c["experts"]
    if s["mask"] is not None:
        x = torch.where(s["mask"][:, None], x, -math.inf)
    scores, p = _scores(x, c["score"])
    key = x
    if s["bias"] is not None:
        # in 64 bits: the choice turns on values next to each other
        key = torch.where(torch.isinf(x), -math.inf, _scores(x.double(), c["score"])[0] + s["bias"].double())
    value, ids = torch.sort(key, dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    chosen = value > -math.inf
    w = torch.where(chosen, scores.gather(1, ids), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    w = w * c["scale"]
    ids = torch.where(chosen, ids, -1)
    if not c["balance"]:
        return ids.to(torch.int32), w, None, None, None, None
    routed = chosen.any(1).sum()
    counts = torch.bincount(ids.flatten() + 1, minlength=E + 1)[1:]
    sums = p.sum(0)
    n = routed.float()
    loss = torch.where(n > 0, E / (k * n * n) * (counts.float() * sums).sum(), 0.0)
    return ids.to(torch.int32), w, counts.to(torch.int32), sums, routed.to(torch.int32), loss


def _route_bwd_plain(s):
    c = s["case"]
    x, E, k = s["logits"].float(), c["experts"], c["top_k"]
    ids, chosen = s["ids"].long().clamp(min=0), s["ids"] >= 0
    there = chosen.any(1, keepdim=True)
    x = torch.where(there, x, -math.inf)
    scores, p = _scores(x, c["score"])
    w = torch.where(chosen, scores.gather(1, ids), 0.0)
    dw = torch.where(chosen, s["dweights"], 0.0) * c["scale"]
    if c["renorm"]:
        total = w.sum(1, keepdim=True).clamp(min=1e-30)
        dw = torch.where(chosen, (dw - (dw * w).sum(1, keepdim=True) / total) / total, 0.0)
    dscore = torch.zeros_like(x).scatter_add_(1, ids, dw)
    if c["score"] == "softmax":
        dx = scores * (dscore - (scores * dscore).sum(1, keepdim=True))
    else:
        dx = dscore * scores * (1 - scores)
    if s["dloss"] is not None:
        n = s["routed"].float()
        f = s["counts"].float() * (s["dloss"] * E / (k * n * n).clamp(min=1))
        dp = p * (f - (p * f).sum(1, keepdim=True))
        dx = dx + (dp if c["score"] == "softmax" else dp * (1 - scores))
    return torch.where(there, dx, 0.0).to(s["logits"].dtype)


def _pow2(e):
    """2 ** e in 64 bits, exactly (|e| < 1022)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x, scale):
    """(values on the E4M3 grid, scales) of x in 64 bits, one scale for each row
    and 128 columns."""
    rows, cols = x.shape
    kb = -(-cols // 128)
    xb = torch.nn.functional.pad(x, (0, 128 * kb - cols)).view(rows, kb, 128)
    amax = xb.abs().amax(2)
    if scale == "pow2":
        m, e = torch.frexp(amax / E4M3_MAX)
        s = _pow2(torch.where(m > 0.5, e, e - 1).clamp(min=-126))
    else:
        s = (amax / E4M3_MAX).float().double()
    s = torch.where(amax > 0, s, 1.0)
    v = xb / s[:, :, None]
    step = _pow2(torch.frexp(v)[1].clamp(min=-5) - 4)
    q = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(rows, 128 * kb)[:, :cols].float(), s.float()


def _rstd(x):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)


def _norm_plain(s):
    c = s["case"]
    # in 64 bits where codes turn on values next to a border
    up = (lambda t: t.double()) if c["out"] != "values" else (lambda t: t.float())
    r, stream = up(s["r"]), None
    if s["y"] is not None:
        z = up(s["y"])
        if s["w_post"] is not None:
            z = z * _rstd(z) * up(s["w_post"])
        if s["gate"] is not None:
            z = z * up(s["gate"])
        r = r + c["alpha"] * z
        stream = r.to(_dtype(c["stream"]))
    n = q = scales = None
    if s["w_pre"] is not None:
        n = r * _rstd(r) * up(s["w_pre"])
        if c["out"] != "values":
            q, scales = _quantise(n, c["scale"])
            q = q.to(torch.float8_e4m3fn)
        n = n.to(_dtype(c["dtype"])) if c["out"] != "codes" else None
    return stream, n, q, scales


def _rms_bwd(d, x, w):
    """Gradients of x and w, and x's normalised rows, from that of x rstd(x) w."""
    r = _rstd(x)
    xh = x * r
    dh = d * w
    return r * (dh - xh * (dh * xh).mean(1, keepdim=True)), (d * xh).sum(0), xh


def _norm_bwd_plain(s):
    c = s["case"]
    dr = s["dr"].float()
    dw_pre = dy = dw_post = dgate = None
    if s["w_pre"] is not None:
        d, dw_pre, _ = _rms_bwd(s["dn"].float(), s["r"].float(), s["w_pre"])
        dr = dr + d
    if s["y"] is not None:
        y, dz = s["y"].float(), dr * c["alpha"]
        z = y if s["w_post"] is None else y * _rstd(y) * s["w_post"]
        if s["gate"] is not None:
            dgate = (dz * z).sum(0) if c["gate"] == "channel" else (dz * z).sum(1, keepdim=True)
            dz = dz * s["gate"]
        if s["w_post"] is not None:
            dz, dw_post, _ = _rms_bwd(dz, y, s["w_post"])
        dy = dz.to(s["y"].dtype)
    return dr.to(s["r"].dtype), dy, dw_post, dgate, dw_pre


def _clip_plain(s):
    c = s["case"]
    # in 64 bits: long sums
    norm = torch.sqrt(sum((g.double() * g.double()).sum() for g in s["grads"]))
    factor = torch.clamp(c["max_norm"] / norm, max=1.0).float()
    return norm.float(), [(g.float() * factor).to(o.dtype) for g, o in zip(s["grads"], s["out"])]


_PLAIN = {"route": _route_plain, "route_bwd": _route_bwd_plain, "norm": _norm_plain, "norm_bwd": _norm_bwd_plain,
          "clip": _clip_plain}


# ---------------------------------------------------------------- the framework's operators

def _route_own(s):
    from moe_grouped_gemm_block_amd import dg
    c = s["case"]
    return tuple(dg.moe_route(s["logits"], c["top_k"], score=c["score"], renormalise=c["renorm"], scale=c["scale"],
                              bias=s["bias"], mask=s["mask"], balance=c["balance"]))


def _route_bwd_own(s):
    from moe_grouped_gemm_block_amd import dg
    c = s["case"]
    return dg.moe_route_bwd(s["dweights"], s["logits"], s["ids"], score=c["score"], renormalise=c["renorm"],
                            scale=c["scale"], dloss=s["dloss"], counts=s["counts"], routed=s["routed"])


def _norm_own(s):
    from moe_grouped_gemm_block_amd import dg
    c = s["case"]
    stream, n, q, scales = dg.residual_norm(s["r"], s["y"], w_post=s["w_post"], gate=s["gate"], alpha=c["alpha"],
                                            w_pre=s["w_pre"], eps=EPS, values=c["out"] != "codes",
                                            codes=None if c["out"] == "values" else c["scale"],
                                            dtype=c["dtype"])
    return stream, n, q if q is None else q.view(torch.float8_e4m3fn), scales


def _norm_bwd_own(s):
    from moe_grouped_gemm_block_amd import dg
    c = s["case"]
    return tuple(dg.residual_norm_bwd(s["dr"], s["dn"], s["r"], s["y"], w_post=s["w_post"], gate=s["gate"],
                                      alpha=c["alpha"], w_pre=s["w_pre"], eps=EPS))


def _clip_own(s):
    from moe_grouped_gemm_block_amd import dg
    norm = dg.grad_norm(s["grads"])
    return norm, dg.clip_grads(s["grads"], norm, s["case"]["max_norm"], out=s["out"])


_OWN = {"route": _route_own, "route_bwd": _route_bwd_own, "norm": _norm_own, "norm_bwd": _norm_bwd_own,
        "clip": _clip_own}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] in ("route", "route_bwd"):
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        n = T * E * size[c["dtype"]] + 8 * T * k + (8 * E + 8 if c["balance"] else 0)
        if c["op"] == "route":
            return {"bytes": n + (T if c["masked"] else 0) + (4 * E if c["bias"] else 0), "flops": 6 * T * E}
        return {"bytes": n + T * E * size[c["dtype"]], "flops": 10 * T * E}
    if c["op"] == "clip":
        n = sum(math.prod(shape) for shape in _shapes(c))
        b = size[c["dtype"]]
        return {"bytes": n * (b + (4 if c["out"] == "f32" else b)), "flops": 3 * n}
    T, H, r, b = c["tokens"], c["hidden"], size[c["stream"]], size[c["dtype"]]
    weights = 4 * H * (c["post"] + c["pre"]) + {"none": 0, "channel": 4 * H, "token": 4 * T}[c["gate"]]
    if c["op"] == "norm":
        out = 0
        if c["pre"]:
            out = (b * H if c["out"] != "codes" else 0) + (H + 4 * -(-H // 128) if c["out"] != "values" else 0)
        return {"bytes": T * (r * H + (b + r) * H * c["block"] + out) + weights,
                "flops": T * H * (8 * c["block"] + 4 * c["pre"])}
    # the stream is read where the norm after it needs it
    return {"bytes": T * H * (2 * r + (r + b) * c["pre"] + 2 * b * c["block"]) + 2 * weights,
            "flops": T * H * (12 * c["block"] + 10 * c["pre"])}


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


def _exact_choice(x, c, bias):
    """Each token's choices, one after another: (ids, which there are)."""
    open_ = x > -math.inf
    left = x
    if bias is not None:
        s = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
        left = torch.where(open_, s + bias.double(), -math.inf)
    left, ids, there = left.clone(), [], []
    for _ in range(c["top_k"]):
        best = left.max(1, keepdim=True).values
        i = (left == best).long().argmax(1, keepdim=True)          # the first of equals
        ids.append(i)
        there.append(best > -math.inf)
        left.scatter_(1, i, -math.inf)
    return torch.cat(ids, 1), torch.cat(there, 1)


def _exact_share(x, ids, there, c):
    """The chosen experts' weights as functions of the logits x, and each token's
    probabilities; logarithms throughout, so that nothing underflows on the way."""
    logs = torch.log_softmax(x, 1) if c["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
    chosen = torch.where(there, logs.gather(1, ids), -math.inf)
    if c["renorm"]:
        chosen = chosen - torch.logsumexp(chosen, 1, keepdim=True)
    p = logs - torch.logsumexp(logs, 1, keepdim=True)
    return c["scale"] * torch.exp(chosen), torch.exp(p)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("route", "route_bwd"):
        x = s["logits"].double()
        rows = (x > -math.inf).any(1) if s["mask"] is None else s["mask"] & (x > -math.inf).any(1)
        E, k, at = c["experts"], c["top_k"], torch.nonzero(rows).flatten()
        n = len(at)
        if c["op"] == "route":
            ids, there = _exact_choice(x[at], c, s["bias"])
            w, p = _exact_share(x[at], ids, there, c)
            weights = torch.zeros(len(x), k, dtype=torch.float64, device="cuda")
            weights[at] = w
            if not c["balance"]:
                return None, weights, None, None, None, None
            sums = p.sum(0)
            share = torch.stack([((ids == e) & there).sum() for e in range(E)]).double() / max(1, k * n)
            return None, weights, None, sums, None, E * (share * sums / max(1, n)).sum()
        # differentiated as it stands, closed experts aside
        dx = torch.zeros_like(x)
        if n:
            xs = x[at].clone().requires_grad_(True)
            ids, there = s["ids"][at].long().clamp(min=0), s["ids"][at] >= 0
            closed = xs.detach() == -math.inf
            safe = torch.where(closed, -1e4, xs)                  # e^-1e4 is 0 in 64 bits too
            w, p = _exact_share(safe, ids, there, c)
            total = (torch.where(there, w, 0.0) * s["dweights"][at].double()).sum()
            if s["dloss"] is not None:
                share = s["counts"].double() / (k * n)
                total = total + s["dloss"].double() * E * (share * p.sum(0) / n).sum()
            dx[at] = torch.autograd.grad(total, xs)[0]
        return dx
    if c["op"] == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        f = min(1.0, c["max_norm"] / norm)
        return torch.tensor(norm, dtype=torch.float64, device="cuda"), [g.double() * f for g in s["grads"]]
    double = lambda t: None if t is None else t.double().clone().requires_grad_(c["op"] == "norm_bwd")
    r, y, w_post, gate, w_pre = (double(s[i]) for i in ("r", "y", "w_post", "gate", "w_pre"))

    def rms(v, w):
        return w * v / v.square().mean(dim=1, keepdim=True).add(EPS).sqrt()

    def after(y, w_post, gate):
        z = y if w_post is None else rms(y, w_post)
        return c["alpha"] * (z if gate is None else gate * z)

    if c["op"] == "norm":
        out = r if y is None else r + after(y, w_post, gate)
        n = q = scales = None
        if w_pre is not None:
            n = rms(out, w_pre)
            if c["out"] != "values":
                q, scales = _exact_codes(n, c["scale"] == "pow2")
        return None if y is None else out, None if c["out"] == "codes" else n, q, scales
    # the stream after the block is what the operator is given as r
    dr = s["dr"].double()
    dw_pre = None
    if w_pre is not None:
        d, dw_pre = torch.autograd.grad((rms(r, w_pre) * s["dn"].double()).sum(), (r, w_pre))
        dr = dr + d
    if y is None:
        return dr, None, None, None, dw_pre
    leaves = [t for t in (y, w_post, gate) if t is not None]
    grads = dict(zip(map(id, leaves), torch.autograd.grad((after(y, w_post, gate) * dr).sum(), leaves)))
    return dr, grads[id(y)], grads.get(id(w_post)), grads.get(id(gate)), dw_pre
