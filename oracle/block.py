"""CPU oracle for the operators that make the mixture-of-experts layer a block of a
model -- TEST INFRASTRUCTURE.  Plain float64 numpy from the operators' definitions.

  route          per-token experts, weights, counts, probability sums, balance loss
  residual_norm  R' = R + alpha gate rms(Y, w_post),  N = rms(R', w_pre)
  clip           g min(1, max_norm / sqrt(sum of squares))

and the gradients.  Beside a gradient stands its mass, the sum of the magnitudes of the
terms it is made of, for bounds on what rounding costs.
"""
from __future__ import annotations

import numpy as np

INF = np.inf


def _sigmoid(x):
    a = np.exp(-np.abs(x))
    return np.where(x > 0, 1.0, a) / (1 + a)


def _log_scores(x, sigmoid):
    """log s of rows of logits, -inf for closed experts."""
    with np.errstate(divide="ignore", invalid="ignore"):
        if sigmoid:
            return np.where(x == -INF, -INF, np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x))))
        m = x.max(1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0)
        z = np.exp(x - m).sum(1, keepdims=True)
        return np.where(x == -INF, -INF, x - m - np.log(np.where(z > 0, z, 1)))


def _shares(logs):
    """e^logs over its row's sum, zeros in rows without an entry."""
    m = logs.max(1, keepdims=True)
    e = np.exp(logs - np.where(np.isfinite(m), m, 0))
    s = e.sum(1, keepdims=True)
    return e / np.where(s > 0, s, 1)


def choose(x, k, sigmoid, bias=None, mask=None):
    """ids [T][k], one token and one choice after another."""
    T, E = x.shape
    logs = _log_scores(x, sigmoid)
    ids = np.full((T, k), -1, np.int64)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        key = x[t].copy() if bias is None else np.where(x[t] == -INF, -INF, np.exp(logs[t]) + bias)
        for j in range(k):
            e = int(np.argmax(key))
            if key[e] == -INF:
                break
            ids[t, j] = e
            key[e] = -INF
    return ids


def route_weights(x, ids, sigmoid, renorm, scale):
    """(weights [T][k], p [T][E]) for the choices `ids`; zeros in rows without one."""
    logs = _log_scores(x, sigmoid)
    there = ids >= 0
    chosen = np.where(there, np.take_along_axis(logs, np.maximum(ids, 0), 1), -INF)
    w = scale * (_shares(chosen) if renorm else np.exp(chosen))
    return np.where(there, w, 0.0), np.where(there.any(1)[:, None], _shares(logs), 0.0)


def route(x, k, sigmoid, renorm, scale, bias=None, mask=None):
    """(ids, weights, counts, prob_sums, routed, loss)."""
    T, E = x.shape
    ids = choose(x, k, sigmoid, bias, mask)
    w, p = route_weights(x, ids, sigmoid, renorm, scale)
    counts = np.bincount(ids[ids >= 0], minlength=E)
    n = int((ids >= 0).any(1).sum())
    sums = p.sum(0)
    return ids, w, counts, sums, n, E / (k * n * n) * float(counts @ sums) if n else 0.0


def route_bwd(dw, x, ids, sigmoid, renorm, scale, dloss=None, counts=None, n=None):
    """(dx, mass): w_j = scale e^(l_j) (over the chosen e^l), l = log s; dl_i/dx_e is
    [i = e] - p_e (softmax) or [i = e] (1 - s_e) (sigmoid)."""
    T, E = x.shape
    k = ids.shape[1]
    there = ids >= 0
    w, p = route_weights(x, ids, sigmoid, renorm, scale)
    dw = np.where(there, dw, 0.0)
    up = w * dw                                               # by log s of the choices
    up_mass = np.abs(up)
    if renorm:
        q = w / scale
        up_mass = up_mass + q * np.abs(up).sum(1, keepdims=True)
        up = up - q * up.sum(1, keepdims=True)
    dl, dl_mass = np.zeros((T, E)), np.zeros((T, E))
    for j in range(k):
        r = np.nonzero(there[:, j])[0]
        np.add.at(dl, (r, ids[r, j]), up[r, j])
        np.add.at(dl_mass, (r, ids[r, j]), up_mass[r, j])
    if not sigmoid and not renorm:
        # (shares among the chosen do not change with a shift of the row)
        dl, dl_mass = dl - p * dl.sum(1, keepdims=True), dl_mass + p * dl_mass.sum(1, keepdims=True)
    if dloss is not None and n:
        g = p * (dloss * E / (k * n * n) * counts)
        dl, dl_mass = dl + g - p * g.sum(1, keepdims=True), dl_mass + np.abs(g) + p * np.abs(g).sum(1, keepdims=True)
    rest = _sigmoid(-x) if sigmoid else 1.0
    dx, mass = dl * rest, dl_mass * rest
    some = there.any(1)[:, None]
    return np.where(some, dx, 0.0), np.where(some, mass, 0.0)


def rstd(x, eps):
    return 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)


def residual_norm(R, Y=None, w_post=None, gate=None, alpha=1.0, w_pre=None, eps=1e-6):
    """(R', N, z): z is what the block adds; N None without w_pre."""
    z = np.zeros_like(R)
    if Y is not None:
        z = Y if w_post is None else Y * rstd(Y, eps) * w_post
        z = alpha * (z if gate is None else z * gate)
    out = R + z
    return out, None if w_pre is None else out * rstd(out, eps) * w_pre, z


def _rms_bwd(e, x, eps):
    """Gradient of x from e, that of x rstd(x), and its mass."""
    r = rstd(x, eps)
    xh = x * r
    return (r * (e - xh * (e * xh).mean(1, keepdims=True)),
            r * (np.abs(e) + np.abs(xh) * np.abs(e * xh).mean(1, keepdims=True)))


def residual_norm_bwd(dR, dN, R, Y=None, w_post=None, gate=None, alpha=1.0, w_pre=None, eps=1e-6):
    """{name: (gradient, mass)} of dR, dY, dw_post, dgate, dw_pre; R is the stream
    after the block, gate [H] or [T][1]."""
    T, H = (R if R is not None else dR).shape
    D, Dm = (np.zeros((T, H)),) * 2 if dR is None else (dR, np.abs(dR))
    out = {}
    if w_pre is not None:
        d, m = _rms_bwd(dN * w_pre, R, eps)
        D, Dm = D + d, Dm + m
        t = dN * R * rstd(R, eps)
        out["dw_pre"] = t.sum(0), np.abs(t).sum(0)
    out["dR"] = D, Dm
    if Y is None:
        return out
    yh = Y if w_post is None else Y * rstd(Y, eps)
    z = yh if w_post is None else yh * w_post
    e, em = alpha * D, abs(alpha) * Dm
    if gate is not None:
        axis, keep = (0, False) if gate.ndim == 1 else (1, True)
        out["dgate"] = (e * z).sum(axis, keepdims=keep), (em * np.abs(z)).sum(axis, keepdims=keep)
        e, em = e * gate, em * np.abs(gate)
    if w_post is not None:
        out["dw_post"] = (e * yh).sum(0), (em * np.abs(yh)).sum(0)
        dy, m = _rms_bwd(e * w_post, Y, eps)
        _, m = _rms_bwd(em * np.abs(w_post), np.abs(Y), eps)
        out["dY"] = dy, m
    else:
        out["dY"] = e, em
    return out


def clip(grads, max_norm):
    """(norm, factor): sums exact to 64 bits."""
    import math
    norm = math.sqrt(math.fsum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / norm) if norm > 0 else 1.0
