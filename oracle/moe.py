"""CPU oracle for the mixture-of-experts operators around the FP8 products --
TEST INFRASTRUCTURE.  Plain float64 numpy from the operators' definitions.

  slot s = t * k + j is token t's j-th choice; expert e's slots, in slot order,
  take rows [o_e, o_e + count_e) of a matrix whose segments are padded to
  `align` rows, the last one to the end
  permute   Y[r] = X[row_slot[r] // k], zeros in padding
  combine   out[t] = sum_j w[t][j] Y[slot_row[t][j]]
  swiglu    a = u g / (1 + exp(-g))
  quantise  one scale per row and 128 columns: the least power of two that
            keeps the block within 448, at least 2^-126 (1 for a zero block)
  wgrad     dW_e = sum over e's rows of dY[r]^T X[r]
"""
from __future__ import annotations

import numpy as np

from .blockscaled import decode_table
from .quantize import encode_nearest

E4M3_MAX = 448.0


def rows_needed(T: int, k: int, G: int, align: int) -> int:
    """The most rows that the segments of T * k slots can take: every expert
    with a slot wastes at most align - 1 rows."""
    used = min(G, T * k)
    return (T * k + (align - 1) * used) // align * align


def sort(ids: np.ndarray, G: int, align: int, M: int):
    """(group_offsets, group_counts, row_slot, slot_row), one slot after another."""
    T, k = ids.shape
    members = [[] for _ in range(G)]
    for s, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < G:
            members[e].append(s)
    offs = np.zeros(G + 1, np.int32)
    row_slot = np.full(M, -1, np.int32)
    slot_row = np.full(T * k, -1, np.int32)
    at = 0
    for e in range(G):
        offs[e] = at
        for i, s in enumerate(members[e]):
            row_slot[at + i] = s
            slot_row[s] = at + i
        at += -(-len(members[e]) // align) * align
    offs[G] = M
    return offs, np.array([len(m) for m in members], np.int32), row_slot, slot_row.reshape(T, k)


def permute(x: np.ndarray, row_slot: np.ndarray, k: int, fill=0) -> np.ndarray:
    out = np.full((len(row_slot),) + x.shape[1:], fill, x.dtype)
    real = row_slot >= 0
    out[real] = x[row_slot[real] // k]
    return out


def combine(y: np.ndarray, slot_row: np.ndarray, w: np.ndarray | None):
    """(out, sum of magnitudes of the terms)."""
    T, k = slot_row.shape
    out, mass = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if slot_row[t, j] >= 0:
                term = (1.0 if w is None else float(w[t, j])) * y[slot_row[t, j]].astype(np.float64)
                out[t] += term
                mass[t] += np.abs(term)
    return out, mass


def combine_bwd(dout: np.ndarray, y: np.ndarray, slot_row: np.ndarray, w: np.ndarray):
    """(dY, dw, sum of magnitudes of dw's terms)."""
    T, k = slot_row.shape
    dy = np.zeros(y.shape)
    dw, mass = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        d = dout[t].astype(np.float64)
        for j in range(k):
            r = slot_row[t, j]
            if r >= 0:
                dy[r] = float(w[t, j]) * d
                terms = d * y[r].astype(np.float64)
                dw[t, j], mass[t, j] = terms.sum(), np.abs(terms).sum()
    return dy, dw, mass


def quantise(x: np.ndarray, pow2: bool):
    """float64 [M][C] -> (codes [M][C], scales float32 [M][ceil(C/128)])."""
    x = np.asarray(x, np.float64)
    M, C = x.shape
    codes = np.zeros((M, C), np.uint8)
    scales = np.ones((M, -(-C // 128)), np.float32)
    for m in range(M):
        for b in range(scales.shape[1]):
            blk = x[m, 128 * b:128 * b + 128]
            amax = float(np.max(np.abs(blk)))
            if amax > 0:
                if pow2:
                    e = -126
                    while amax > E4M3_MAX * 2.0 ** e:
                        e += 1
                    scales[m, b] = 2.0 ** e
                else:
                    scales[m, b] = np.float32(amax / E4M3_MAX)
            codes[m, 128 * b:128 * b + 128] = encode_nearest(blk / np.float64(scales[m, b]))
    return codes, scales


def dequantise(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    C = codes.shape[1]
    return decode_table()[codes] * np.repeat(scales.astype(np.float64), 128, axis=1)[:, :C]


def swiglu(g: np.ndarray, u: np.ndarray) -> np.ndarray:
    g, u = g.astype(np.float64), u.astype(np.float64)
    return u * (g / (1 + np.exp(-g)))


def swiglu_bwd(da: np.ndarray, g: np.ndarray, u: np.ndarray):
    """(dg, du, magnitude of dg's terms)."""
    da, g, u = (v.astype(np.float64) for v in (da, g, u))
    p = 1 / (1 + np.exp(-g))
    return (da * u * p * (1 + g * (1 - p)), da * g * p, np.abs(da * u) * p * (1 + np.abs(g) * (1 - p)))


def wgrad(dy: np.ndarray, x: np.ndarray, offs: np.ndarray, counts: np.ndarray):
    """(dW, sum of magnitudes of its terms)."""
    G = len(counts)
    dw = np.zeros((G, dy.shape[1], x.shape[1]))
    mass = np.zeros_like(dw)
    for e in range(G):
        r = slice(offs[e], offs[e] + counts[e])
        d, v = dy[r].astype(np.float64), x[r].astype(np.float64)
        dw[e], mass[e] = d.T @ v, np.abs(d).T @ np.abs(v)
    return dw, mass
