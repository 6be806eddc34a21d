"""ctypes binding of libdg.so (argument marshalling only).

The functions named like the C entry points take raw integers (device
addresses, sizes, a hipStream_t handle) and return the dg_status code.  The
torch-facing helpers below them only check dtypes / shapes / devices, pass
``data_ptr()`` values and the current stream, and raise on a non-zero status;
every step of the computation runs in the library's HIP kernels.  For the
mixture-of-experts operators that part is native code (_dg_torch).

Loading fails loudly when the library has not been built: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("DG_LIBRARY", os.path.join(_PKG, "libdg.so"))

DG_OUT_F32 = 0
DG_OUT_BF16 = 1
DG_IN_F32 = 0
DG_IN_BF16 = 1
DG_FP8_E4M3 = 0
DG_FP8_E5M2 = 1
DG_IDX_I32 = 0
DG_IDX_I64 = 1
DG_SCALE_AMAX = 0
DG_SCALE_POW2 = 1
DG_SCORE_SOFTMAX = 0
DG_SCORE_SIGMOID = 1
DG_GATE_NONE = 0
DG_GATE_CHANNEL = 1
DG_GATE_TOKEN = 2
DG_OK = 0
DG_ERR_INVALID_ARG = -1
DG_ERR_UNSUPPORTED = -2
DG_ERR_LAUNCH = -3

EXPORTED = ("dg_gemm_fp8_blockscaled", "dg_grouped_gemm_fp8", "dg_gemm_fp8_ex", "dg_gemm_fp8_ex_noalloc",
            "dg_grouped_gemm_fp8_ex", "dg_grouped_gemm_fp8_ex_counts", "dg_grouped_gemm_fp8_segments",
            "dg_quantize_fp8_blockscaled", "dg_moe_sort", "dg_moe_rows", "dg_moe_sort_workspace",
            "dg_moe_permute", "dg_moe_permute_fp8", "dg_moe_combine", "dg_moe_combine_bwd", "dg_swiglu_fp8",
            "dg_swiglu_fp8_bwd", "dg_grouped_wgrad_fp8", "dg_moe_route", "dg_moe_route_workspace", "dg_moe_route_bwd",
            "dg_residual_norm", "dg_residual_norm_bwd", "dg_residual_norm_bwd_workspace", "dg_grad_norm",
            "dg_grad_norm_workspace", "dg_clip_grads", "dg_status_string")

_lib = None


def lib() -> ctypes.CDLL:
    """Load libdg.so once; raise if it is missing.

    torch is imported first when it is installed: torch's ROCm build carries
    its own HIP runtime, and libdg.so's dependency on the HIP runtime is then
    satisfied by that already-loaded copy.  Loaded the other way round, the
    process would hold two HIP runtimes (the system one for libdg.so, torch's
    for the tensors), and the library's runtime, initialised second, cannot
    use the GPU (its device queries fail).
    """
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m moe_grouped_gemm_block_amd.build` "
                "(there is no non-HIP fallback)")
        try:
            import torch  # noqa: F401  (one HIP runtime for torch and the library)
        except ImportError:
            pass
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, ci, cf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        L.dg_gemm_fp8_blockscaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
        L.dg_gemm_fp8_blockscaled.restype = ci
        L.dg_grouped_gemm_fp8.argtypes = [vp, vp, vp, vp, vp, vp, ci, i64, i64, i64, ci, vp]
        L.dg_grouped_gemm_fp8.restype = ci
        L.dg_gemm_fp8_ex.argtypes = [vp, ci, vp, ci, vp, ci, vp, vp, i64, i64, i64, ci, vp]
        L.dg_gemm_fp8_ex.restype = ci
        L.dg_gemm_fp8_ex_noalloc.argtypes = [vp, ci, vp, ci, vp, ci, vp, vp, i64, i64, i64, ci, vp]
        L.dg_gemm_fp8_ex_noalloc.restype = ci
        L.dg_grouped_gemm_fp8_ex.argtypes = [vp, ci, vp, ci, vp, ci, vp, vp, vp, ci, i64, i64, i64, ci, vp]
        L.dg_grouped_gemm_fp8_ex.restype = ci
        L.dg_grouped_gemm_fp8_ex_counts.argtypes = [vp, ci, vp, ci, vp, ci, vp, vp, vp, vp, ci, i64, i64, i64,
                                                    ci, vp]
        L.dg_grouped_gemm_fp8_ex_counts.restype = ci
        L.dg_grouped_gemm_fp8_segments.argtypes = [vp, ci, vp, vp, ci, vp, vp, vp, ci, i64, i64, i64, ci, vp]
        L.dg_grouped_gemm_fp8_segments.restype = ci
        L.dg_quantize_fp8_blockscaled.argtypes = [vp, ci, vp, vp, i64, i64, ci, vp]
        L.dg_quantize_fp8_blockscaled.restype = ci
        around = {
            "dg_moe_sort": (ci, [vp, ci, i64, ci, ci, ci, i64, vp, vp, vp, vp, vp, vp]),
            "dg_moe_rows": (i64, [i64, ci, ci, ci]),
            "dg_moe_sort_workspace": (i64, [i64, ci, ci]),
            "dg_moe_permute": (ci, [vp, ci, vp, vp, vp, i64, ci, i64, i64, vp]),
            "dg_moe_permute_fp8": (ci, [vp, ci, vp, vp, ci, vp, vp, i64, ci, i64, i64, vp]),
            "dg_moe_combine": (ci, [vp, ci, vp, vp, vp, i64, ci, i64, i64, vp]),
            "dg_moe_combine_bwd": (ci, [vp, vp, ci, vp, vp, vp, vp, vp, i64, ci, i64, i64, vp]),
            "dg_swiglu_fp8": (ci, [vp, ci, vp, vp, vp, vp, i64, i64, vp]),
            "dg_swiglu_fp8_bwd": (ci, [vp, ci, vp, vp, vp, i64, i64, vp]),
            "dg_grouped_wgrad_fp8": (ci, [vp, vp, vp, vp, vp, ci, i64, i64, i64, vp, ci, ci, vp]),
            "dg_moe_route": (ci, [vp, ci, vp, vp, i64, i64, ci, ci, ci, cf, vp, vp, vp, vp, vp, vp, vp, vp]),
            "dg_moe_route_workspace": (i64, [i64, i64, ci]),
            "dg_moe_route_bwd": (ci, [vp, vp, ci, vp, vp, vp, vp, i64, i64, ci, ci, ci, cf, vp, vp]),
            "dg_residual_norm": (ci, [vp, ci, vp, ci, vp, vp, ci, cf, vp, cf, vp, vp, vp, vp, ci, i64, i64, vp]),
            "dg_residual_norm_bwd": (ci, [vp, vp, vp, ci, vp, ci, vp, vp, ci, cf, vp, cf, vp, vp, vp, vp, vp, i64,
                                          i64, vp, vp]),
            "dg_residual_norm_bwd_workspace": (i64, [i64, i64, ci]),
            "dg_grad_norm": (ci, [vp, vp, vp, ci, vp, vp, vp]),
            "dg_grad_norm_workspace": (i64, [vp, vp, ci]),
            "dg_clip_grads": (ci, [vp, vp, vp, ci, vp, cf, vp, vp, vp]),
        }
        for name, (result, arguments) in around.items():
            if hasattr(L, name):                  # a library of an earlier build may lack it; calling it then raises
                getattr(L, name).restype, getattr(L, name).argtypes = result, arguments
        L.dg_status_string.argtypes = [ci]
        L.dg_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


# ---------------------------------------------------------------- raw C names

def dg_gemm_fp8_blockscaled(A, sA, B, sB, C, M, N, K, out_dtype, stream) -> int:
    return lib().dg_gemm_fp8_blockscaled(A, sA, B, sB, C, M, N, K, out_dtype, stream)


def dg_grouped_gemm_fp8(A, sA, B, sB, C, group_offsets, num_groups, M_total, N, K,
                        out_dtype, stream) -> int:
    return lib().dg_grouped_gemm_fp8(A, sA, B, sB, C, group_offsets, num_groups, M_total,
                                     N, K, out_dtype, stream)


def dg_gemm_fp8_ex(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, M, N, K, out_dtype, stream) -> int:
    return lib().dg_gemm_fp8_ex(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, M, N, K, out_dtype, stream)


def dg_gemm_fp8_ex_noalloc(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, M, N, K, out_dtype, stream) -> int:
    return lib().dg_gemm_fp8_ex_noalloc(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, M, N, K, out_dtype, stream)


def dg_grouped_gemm_fp8_ex(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, group_offsets, num_groups, M_total,
                           N, K, out_dtype, stream) -> int:
    return lib().dg_grouped_gemm_fp8_ex(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, group_offsets, num_groups,
                                        M_total, N, K, out_dtype, stream)


def dg_grouped_gemm_fp8_ex_counts(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, group_offsets, group_counts,
                                  num_groups, M_total, N, K, out_dtype, stream) -> int:
    return lib().dg_grouped_gemm_fp8_ex_counts(A, a_fmt, sA, sa_rows, B, b_fmt, sB, C, group_offsets,
                                               group_counts, num_groups, M_total, N, K, out_dtype, stream)


def dg_grouped_gemm_fp8_segments(A, a_fmt, sA, B, b_fmt, sB, C, group_offsets, num_groups, M_total, N, K,
                                 out_dtype, stream) -> int:
    return lib().dg_grouped_gemm_fp8_segments(A, a_fmt, sA, B, b_fmt, sB, C, group_offsets, num_groups,
                                              M_total, N, K, out_dtype, stream)


def dg_quantize_fp8_blockscaled(X, in_dtype, Q, S, M, K, block_rows, stream) -> int:
    return lib().dg_quantize_fp8_blockscaled(X, in_dtype, Q, S, M, K, block_rows, stream)


def dg_moe_sort(ids, ids_dtype, T, top_k, num_groups, align, M_total, group_offsets, group_counts, row_slot,
                slot_row, workspace, stream) -> int:
    return lib().dg_moe_sort(ids, ids_dtype, T, top_k, num_groups, align, M_total, group_offsets, group_counts,
                             row_slot, slot_row, workspace, stream)


def dg_moe_rows(T, top_k, num_groups, align) -> int:
    return lib().dg_moe_rows(T, top_k, num_groups, align)


def dg_moe_sort_workspace(T, top_k, num_groups) -> int:
    return lib().dg_moe_sort_workspace(T, top_k, num_groups)


def dg_moe_permute(X, dtype, Y, slot_row, row_slot, T, top_k, M_total, H, stream) -> int:
    return lib().dg_moe_permute(X, dtype, Y, slot_row, row_slot, T, top_k, M_total, H, stream)


def dg_moe_permute_fp8(X, in_dtype, Q, S, scale_mode, slot_row, row_slot, T, top_k, M_total, H, stream) -> int:
    return lib().dg_moe_permute_fp8(X, in_dtype, Q, S, scale_mode, slot_row, row_slot, T, top_k, M_total, H,
                                    stream)


def dg_moe_combine(Y, dtype, weights, slot_row, out, T, top_k, M_total, H, stream) -> int:
    return lib().dg_moe_combine(Y, dtype, weights, slot_row, out, T, top_k, M_total, H, stream)


def dg_moe_combine_bwd(dOut, Y, dtype, weights, slot_row, row_slot, dY, dweights, T, top_k, M_total, H,
                       stream) -> int:
    return lib().dg_moe_combine_bwd(dOut, Y, dtype, weights, slot_row, row_slot, dY, dweights, T, top_k, M_total,
                                    H, stream)


def dg_swiglu_fp8(H, in_dtype, A, sA, Hq, sH, M, I, stream) -> int:
    return lib().dg_swiglu_fp8(H, in_dtype, A, sA, Hq, sH, M, I, stream)


def dg_swiglu_fp8_bwd(dA, dtype, Hq, sH, dH, M, I, stream) -> int:
    return lib().dg_swiglu_fp8_bwd(dA, dtype, Hq, sH, dH, M, I, stream)


def dg_grouped_wgrad_fp8(dY, X, sX, group_offsets, group_counts, num_groups, M_total, N, K, dW, out_dtype,
                         accumulate, stream) -> int:
    return lib().dg_grouped_wgrad_fp8(dY, X, sX, group_offsets, group_counts, num_groups, M_total, N, K, dW,
                                      out_dtype, accumulate, stream)


def dg_moe_route(logits, dtype, bias, mask, T, E, top_k, score, renormalise, scale, ids, weights, counts, prob_sums,
                 routed, loss, workspace, stream) -> int:
    return lib().dg_moe_route(logits, dtype, bias, mask, T, E, top_k, score, renormalise, scale, ids, weights, counts,
                              prob_sums, routed, loss, workspace, stream)


def dg_moe_route_workspace(T, E, top_k) -> int:
    return lib().dg_moe_route_workspace(T, E, top_k)


def dg_moe_route_bwd(dweights, logits, dtype, ids, counts, routed, dloss, T, E, top_k, score, renormalise, scale,
                     dlogits, stream) -> int:
    return lib().dg_moe_route_bwd(dweights, logits, dtype, ids, counts, routed, dloss, T, E, top_k, score, renormalise,
                                  scale, dlogits, stream)


def dg_residual_norm(R, r_dtype, Y, dtype, w_post, gate, gate_kind, alpha, w_pre, eps, R_out, N, Q, S, scale_mode, T, H,
                     stream) -> int:
    return lib().dg_residual_norm(R, r_dtype, Y, dtype, w_post, gate, gate_kind, alpha, w_pre, eps, R_out, N, Q, S,
                                  scale_mode, T, H, stream)


def dg_residual_norm_bwd(dR, dN, R, r_dtype, Y, dtype, w_post, gate, gate_kind, alpha, w_pre, eps, dR_out, dY, dw_post,
                         dgate, dw_pre, T, H, workspace, stream) -> int:
    return lib().dg_residual_norm_bwd(dR, dN, R, r_dtype, Y, dtype, w_post, gate, gate_kind, alpha, w_pre, eps, dR_out,
                                      dY, dw_post, dgate, dw_pre, T, H, workspace, stream)


def dg_residual_norm_bwd_workspace(T, H, sums) -> int:
    return lib().dg_residual_norm_bwd_workspace(T, H, sums)


def dg_grad_norm(grads, sizes, dtypes, count, norm, workspace, stream) -> int:
    """grads, sizes, dtypes: ctypes arrays of host memory."""
    return lib().dg_grad_norm(grads, sizes, dtypes, count, norm, workspace, stream)


def dg_grad_norm_workspace(sizes, dtypes, count) -> int:
    return lib().dg_grad_norm_workspace(sizes, dtypes, count)


def dg_clip_grads(grads, sizes, dtypes, count, norm, max_norm, outs, out_dtypes, stream) -> int:
    return lib().dg_clip_grads(grads, sizes, dtypes, count, norm, max_norm, outs, out_dtypes, stream)


def dg_status_string(status: int) -> str:
    return lib().dg_status_string(status).decode()


class DGError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {dg_status_string(status)} ({status})")
        self.status = status


# ---------------------------------------------------------------- torch helpers

def _torch():
    import torch
    return torch


def _check_fp8(t, name):
    torch = _torch()
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2):
        raise TypeError(f"{name} must be uint8 FP8 codes, float8_e4m3fn or float8_e5m2, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")


def operand_fmt(t, fmt, name) -> int:
    """FP8 format code of operand tensor t.  A float8 dtype names its format;
    uint8 codes take `fmt` ("e4m3" when None).  An explicit `fmt` that
    disagrees with a float8 dtype is an error (the bytes would otherwise be
    decoded in the wrong format)."""
    torch = _torch()
    implied = {torch.float8_e4m3fn: DG_FP8_E4M3, torch.float8_e5m2: DG_FP8_E5M2}.get(t.dtype)
    if fmt is None:
        return DG_FP8_E4M3 if implied is None else implied
    code = fmt_code(fmt)
    if implied is not None and code != implied:
        raise ValueError(f"{name} is {t.dtype} but its format is given as {fmt!r}")
    return code


def _check_f32(t, name, shape):
    torch = _torch()
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 device tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _out(C, rows, N, out_dtype, like):
    torch = _torch()
    dt = torch.float32 if out_dtype == DG_OUT_F32 else torch.bfloat16
    if C is None:
        return torch.empty((rows, N), dtype=dt, device=like.device)
    if C.dtype != dt or tuple(C.shape) != (rows, N) or not C.is_contiguous():
        raise ValueError("C has the wrong dtype, shape or layout")
    return C


def out_code(out_dtype) -> int:
    if out_dtype in (DG_OUT_F32, "f32", "float32"):
        return DG_OUT_F32
    if out_dtype in (DG_OUT_BF16, "bf16", "bfloat16"):
        return DG_OUT_BF16
    raise ValueError(f"unknown out_dtype {out_dtype!r}")


def fmt_code(fmt) -> int:
    if fmt in (DG_FP8_E4M3, "e4m3"):
        return DG_FP8_E4M3
    if fmt in (DG_FP8_E5M2, "e5m2"):
        return DG_FP8_E5M2
    raise ValueError(f"unknown FP8 format {fmt!r}")


def _stream(stream):
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _sa_rows(sA, M, K):
    """Rows per A scale block implied by sA's shape: 128 ([ceil(M/128)][K/128])
    or 1 ([M][K/128]); the first wins where both fit (M <= 1)."""
    if tuple(sA.shape) == (-(-M // 128), -(-K // 128)):
        return 128
    if tuple(sA.shape) == (M, -(-K // 128)):
        return 1
    raise ValueError(f"sA has shape {tuple(sA.shape)}; expected {(-(-M // 128), -(-K // 128))} "
                     f"(128 x 128 blocks) or {(M, -(-K // 128))} (1 x 128 blocks)")


def gemm_fp8_blockscaled(A, sA, B, sB, out_dtype="bf16", C=None, stream=None, a_fmt=None, b_fmt=None):
    """C[M][N] = block-scaled A[M][K] x B (stored [N][K]) on the device; the
    operands' FP8 formats are "e4m3" or "e5m2" (None: from a float8 dtype,
    E4M3 for uint8 codes).  sA holds one scale per 128 x 128 block
    ([ceil(M/128)][K/128]) or per row and 128 columns ([M][K/128])."""
    _check_fp8(A, "A")
    _check_fp8(B, "B")
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError("A and B must share K")
    rows = _sa_rows(sA, M, K)
    _check_f32(sA, "sA", tuple(sA.shape))
    _check_f32(sB, "sB", (-(-N // 128), -(-K // 128)))
    code = out_code(out_dtype)
    C = _out(C, M, N, code, A)
    fa, fb = operand_fmt(A, a_fmt, "A"), operand_fmt(B, b_fmt, "B")
    if fa == DG_FP8_E4M3 and fb == DG_FP8_E4M3 and rows == 128:
        st = dg_gemm_fp8_blockscaled(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(),
                                     C.data_ptr(), M, N, K, code, _stream(stream))
    else:
        st = dg_gemm_fp8_ex(A.data_ptr(), fa, sA.data_ptr(), rows, B.data_ptr(), fb, sB.data_ptr(),
                            C.data_ptr(), M, N, K, code, _stream(stream))
    if st != DG_OK:
        raise DGError(st, "dg_gemm_fp8_blockscaled")
    return C


def grouped_gemm_fp8(A, sA, B, sB, group_offsets, out_dtype="bf16", C=None, stream=None,
                     a_fmt=None, b_fmt=None, group_counts=None):
    """MoE grouped GEMM over contiguous 128-row-padded expert segments.
    group_counts (device int32 [G], optional): real rows per expert; the
    padding rows after them come out as zeros and skip the work where whole
    wave sub-tiles are padding (dg_grouped_gemm_fp8_ex_counts)."""
    torch = _torch()
    _check_fp8(A, "A")
    _check_fp8(B, "B")
    M_total, K = A.shape
    G, N, K2 = B.shape
    if K != K2:
        raise ValueError("A and B must share K")
    rows = _sa_rows(sA, M_total, K)
    _check_f32(sA, "sA", tuple(sA.shape))
    _check_f32(sB, "sB", (G, -(-N // 128), -(-K // 128)))
    if (group_offsets.dtype != torch.int32 or not group_offsets.is_cuda
            or tuple(group_offsets.shape) != (G + 1,)):
        raise ValueError("group_offsets must be a device int32 tensor of G + 1 entries")
    code = out_code(out_dtype)
    C = _out(C, M_total, N, code, A)
    fa, fb = operand_fmt(A, a_fmt, "A"), operand_fmt(B, b_fmt, "B")
    if group_counts is not None:
        if (group_counts.dtype != torch.int32 or not group_counts.is_cuda
                or tuple(group_counts.shape) != (G,)):
            raise ValueError("group_counts must be a device int32 tensor of G entries")
        st = dg_grouped_gemm_fp8_ex_counts(A.data_ptr(), fa, sA.data_ptr(), rows, B.data_ptr(), fb,
                                           sB.data_ptr(), C.data_ptr(), group_offsets.data_ptr(),
                                           group_counts.data_ptr(), G, M_total, N, K, code, _stream(stream))
    elif fa == DG_FP8_E4M3 and fb == DG_FP8_E4M3 and rows == 128:
        st = dg_grouped_gemm_fp8(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(),
                                 C.data_ptr(), group_offsets.data_ptr(), G, M_total, N, K, code,
                                 _stream(stream))
    else:
        st = dg_grouped_gemm_fp8_ex(A.data_ptr(), fa, sA.data_ptr(), rows, B.data_ptr(), fb, sB.data_ptr(),
                                    C.data_ptr(), group_offsets.data_ptr(), G, M_total, N, K, code,
                                    _stream(stream))
    if st != DG_OK:
        raise DGError(st, "dg_grouped_gemm_fp8")
    return C


def grouped_gemm_fp8_segments(A, sA, B, sB, group_offsets, out_dtype="bf16", C=None, stream=None,
                              a_fmt=None, b_fmt=None):
    """MoE grouped GEMM over packed (unpadded) expert segments with one A
    scale per row, sA [M_total][K/128]; meant for few rows per expert."""
    torch = _torch()
    _check_fp8(A, "A")
    _check_fp8(B, "B")
    M_total, K = A.shape
    G, N, K2 = B.shape
    if K != K2:
        raise ValueError("A and B must share K")
    _check_f32(sA, "sA", (M_total, -(-K // 128)))
    _check_f32(sB, "sB", (G, -(-N // 128), -(-K // 128)))
    if (group_offsets.dtype != torch.int32 or not group_offsets.is_cuda
            or tuple(group_offsets.shape) != (G + 1,)):
        raise ValueError("group_offsets must be a device int32 tensor of G + 1 entries")
    code = out_code(out_dtype)
    C = _out(C, M_total, N, code, A)
    st = dg_grouped_gemm_fp8_segments(A.data_ptr(), operand_fmt(A, a_fmt, "A"), sA.data_ptr(), B.data_ptr(),
                                      operand_fmt(B, b_fmt, "B"), sB.data_ptr(), C.data_ptr(), group_offsets.data_ptr(),
                                      G, M_total, N, K, code, _stream(stream))
    if st != DG_OK:
        raise DGError(st, "dg_grouped_gemm_fp8_segments")
    return C


def quantize_fp8_blockscaled(X, block_rows=128, Q=None, S=None, stream=None):
    """E4M3 codes and FP32 block scales of X[M][K] (float32 or bfloat16), one
    scale per block_rows x 128 block (block_rows = 128 or 1)."""
    torch = _torch()
    if X.dtype == torch.float32:
        code = DG_IN_F32
    elif X.dtype == torch.bfloat16:
        code = DG_IN_BF16
    else:
        raise TypeError(f"X must be float32 or bfloat16, got {X.dtype}")
    if not X.is_cuda or not X.is_contiguous() or X.dim() != 2:
        raise ValueError("X must be a contiguous 2-D device tensor")
    M, K = X.shape
    if Q is None:
        Q = torch.empty((M, K), dtype=torch.uint8, device=X.device)
    if S is None:
        S = torch.empty((-(-M // block_rows), K // 128), dtype=torch.float32, device=X.device)
    _check_fp8(Q, "Q")
    _check_f32(S, "S", (-(-M // block_rows), K // 128))
    if tuple(Q.shape) != (M, K):
        raise ValueError("Q must have the shape of X")
    st = dg_quantize_fp8_blockscaled(X.data_ptr(), code, Q.data_ptr(), S.data_ptr(), M, K, block_rows,
                                     _stream(stream))
    if st != DG_OK:
        raise DGError(st, "dg_quantize_fp8_blockscaled")
    return Q, S


# ---------------------------------------------------------------- around the products
#
# Checks of the tensors, output tensors and the current stream are native code
# (csrc/binding.cpp, the module _dg_torch), which then makes the calls above.  Like
# the helpers above, these record nothing for autograd: outputs are detached, and a
# layer calls the forward and backward operators itself (examples/moe_layer.py).

class MoEPlan(NamedTuple):
    """What moe_sort finds out about one batch (device int32 tensors)."""
    group_offsets: object     # [G + 1] first rows of the experts' segments; the last entry is the row count
    group_counts: object      # [G] real rows
    row_slot: object          # [M] slot t * top_k + j of a row, -1 for padding
    slot_row: object          # [T][top_k] row of a slot, -1 when dropped


_binding = None


def binding():
    """The native binding, loaded on first use; raise if it is missing."""
    global _binding
    if _binding is None:
        lib()                                     # torch's HIP runtime first, see there
        _torch()
        try:
            from . import _dg_torch
        except ImportError as e:
            raise RuntimeError(f"{_PKG}/_dg_torch.so cannot be loaded ({e}); "
                               f"run `python -m moe_grouped_gemm_block_amd.build` on a machine with ROCm") from e
        _dg_torch.load(LIB_PATH, DGError)
        _binding = _dg_torch
    return _binding


def _on(stream):
    """Context in which `stream` (a Stream or its handle) is the current one:
    new tensors then belong to it, so that the allocator never hands out memory
    that other streams' pending work still uses."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _call(name, stream, *args):
    f = getattr(_binding or binding(), name)
    if stream is None:
        return f(*args)
    with _on(stream):
        return f(*args)


def moe_sort(ids, num_groups, align=128, rows=None, stream=None):
    """The MoEPlan of expert ids[T][top_k] (int32 or int64; a choice whose id
    lies outside [0, num_groups) is dropped).  align: 128 for the padded
    segments of grouped_gemm_fp8, 1 for the packed ones of
    grouped_gemm_fp8_segments.  rows: rows of the sorted matrix, by default the
    most that any ids need (dg_moe_rows); nothing waits for the device."""
    return MoEPlan(*_call("moe_sort", stream, ids, num_groups, align, rows))


def moe_permute(X, slot_row, row_slot, Y=None, stream=None):
    """Rows of X[T][H] (bfloat16 or float32) in the plan's order: Y[M][H], zeros
    in rows of padding.  Its gradient is moe_combine without weights."""
    return _call("moe_permute", stream, X, slot_row, row_slot, Y)


def scale_code(scale) -> int:
    if scale in (DG_SCALE_AMAX, "amax"):
        return DG_SCALE_AMAX
    if scale in (DG_SCALE_POW2, "pow2"):
        return DG_SCALE_POW2
    raise ValueError(f"unknown scale mode {scale!r}")


def moe_permute_fp8(X, slot_row, row_slot, scale="pow2", Q=None, S=None, stream=None):
    """The same, quantised: E4M3 codes Q[M][H] and one FP32 scale per row and 128
    columns, S[M][ceil(H/128)] (A and sA of the grouped products).  scale:
    "pow2" (powers of two: what grouped_wgrad_fp8 reads without rounding) or
    "amax" (amax / 448)."""
    return _call("moe_permute_fp8", stream, X, slot_row, row_slot, scale_code(scale), Q, S)


def moe_combine(Y, slot_row, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t][j] Y[slot_row[t][j]] (weights None: ones), of Y's
    dtype; dropped choices add nothing."""
    return _call("moe_combine", stream, Y, slot_row, weights, out)


def moe_combine_bwd(dOut, Y, slot_row, row_slot, weights, dY=None, dweights=None, stream=None):
    """The gradient of moe_combine with weights: dY[M][H] (zeros in rows of
    padding) and dweights[T][top_k] (float32)."""
    return _call("moe_combine_bwd", stream, dOut, Y, slot_row, row_slot, weights, dY, dweights)


def swiglu_fp8(H, checkpoint=True, stream=None):
    """a = u g / (1 + exp(-g)) of H[M][2 I] = [g | u] (bfloat16 or float32) in 8
    bits: (A[M][I], sA[M][ceil(I/128)], Hq[M][2 I], sH[M][2][ceil(I/128)]), E4M3
    codes with power-of-two scales.  Hq, sH are H's checkpoint for
    swiglu_fp8_bwd; None without `checkpoint`.  sA and sH share an allocation."""
    return _call("swiglu_fp8", stream, H, checkpoint)


def swiglu_fp8_bwd(dA, Hq, sH, dH=None, stream=None):
    """The gradient dH[M][2 I] of swiglu_fp8 from dA[M][I] (bfloat16 or float32)
    and the checkpoint."""
    return _call("swiglu_fp8_bwd", stream, dA, Hq, sH, dH)


def grouped_wgrad_fp8(dY, X, sX, group_offsets, group_counts=None, out_dtype="f32", dW=None, accumulate=False,
                      stream=None):
    """dW[G][N][K], each expert's dY^T X over its rows, of dY[M][N] (bfloat16) and
    8-bit activations X[M][K] with scales sX[M][ceil(K/128)].  accumulate adds to
    dW; rows past group_counts are not used."""
    return _call("grouped_wgrad_fp8", stream, dY, X, sX, group_offsets, group_counts, out_code(out_dtype), dW,
                 accumulate)


# ---------------------------------------------------------------- around a block of a model

class MoERoute(NamedTuple):
    """What moe_route finds out about one batch.  The last four are None without
    `balance`; routed and loss have no dimensions."""
    ids: object               # int32 [T][top_k], -1: no expert
    weights: object           # float32 [T][top_k]
    counts: object            # int32 [E] tokens that chose an expert
    prob_sums: object         # float32 [E] the tokens' probabilities added up
    routed: object            # int32 tokens with a choice
    loss: object              # float32 balance loss


class ResidualNorm(NamedTuple):
    R: object                 # [T][H] the stream after the block, None without one
    N: object                 # [T][H] its norm, None without `values` or w_pre
    Q: object                 # uint8 [T][H] the norm's E4M3 codes, None without `codes`
    S: object                 # float32 [T][ceil(H/128)] their scales


class ResidualNormGrads(NamedTuple):
    """None for what the forward call did not have."""
    dR: object                # [T][H] of the stream before the block
    dY: object                # [T][H]
    dw_post: object           # float32 [H]
    dgate: object             # float32, of gate's shape
    dw_pre: object            # float32 [H]


def score_code(score) -> int:
    if score in (DG_SCORE_SOFTMAX, "softmax"):
        return DG_SCORE_SOFTMAX
    if score in (DG_SCORE_SIGMOID, "sigmoid"):
        return DG_SCORE_SIGMOID
    raise ValueError(f"unknown score {score!r}")


def moe_route(logits, top_k, score="softmax", renormalise=True, scale=1.0, bias=None, mask=None, balance=True,
              stream=None):
    """The MoERoute of router logits[T][E] (float32 or bfloat16; -inf closes an expert
    to a token): each token's top_k experts, largest first, and their weights,
    scale s_j, with `renormalise` divided by the chosen scores' sum.  score:
    "softmax" or "sigmoid".  bias float32 [E] is added to the scores for the choice
    alone.  mask bool [T]: False for rows that hold no token.  balance: also the
    experts' load and the balance loss E / (top_k n^2) sum counts_e prob_sums_e."""
    return MoERoute(*_call("moe_route", stream, logits, top_k, score_code(score), renormalise, scale, bias, mask,
                           balance))


def moe_route_bwd(dweights, logits, ids, score="softmax", renormalise=True, scale=1.0, dloss=None, counts=None,
                  routed=None, dlogits=None, stream=None):
    """The gradient of the logits from dweights[T][top_k] (float32) and dloss (a
    float32 tensor of one element, with moe_route's counts and routed, or their sums
    over several devices)."""
    return _call("moe_route_bwd", stream, dweights, logits, ids, score_code(score), renormalise, scale, dloss, counts,
                 routed, dlogits)


def _dtype_code(dtype):
    torch = _torch()
    if dtype in (None, "bf16", "bfloat16", torch.bfloat16):
        return DG_IN_BF16
    if dtype in ("f32", "float32", torch.float32):
        return DG_IN_F32
    raise ValueError(f"unknown dtype {dtype!r}")


def residual_norm(R, Y=None, w_post=None, gate=None, alpha=1.0, w_pre=None, eps=1e-6, values=True, codes=None,
                  dtype=None, stream=None):
    """The residual stream R[T][H] past a block with output Y[T][H], and the norm before
    the next one: R' = R + alpha gate rms(Y, w_post), N = rms(R', w_pre), with
    rms(v, w) = w v / sqrt(mean(v^2) + eps).  Weights are float32 [H]; gate float32,
    [H] by channel or [T][1] by token.  R and Y are float32 or bfloat16, each its own.
    Y None: no block before (R' is R).  w_post None: Y as it is.  w_pre None: no norm.
    values: N as values of `dtype` (Y's; without Y bfloat16 if None); codes: "pow2" or
    "amax": also as E4M3 codes with a scale per row and 128 columns, A and sA of the
    products."""
    mode = -1 if codes is None else scale_code(codes)
    code = -1 if Y is not None and dtype is None else _dtype_code(dtype)
    return ResidualNorm(*_call("residual_norm", stream, R, Y, w_post, gate, alpha, w_pre, eps, values, mode, code))


def residual_norm_bwd(dR, dN, R, Y=None, w_post=None, gate=None, alpha=1.0, w_pre=None, eps=1e-6, stream=None):
    """The ResidualNormGrads of residual_norm from the gradients dR of R' (None: zeros)
    and dN of N (None without w_pre).  R is the stream that the forward call returned,
    R' (its input where there was no block); without w_pre it may be None."""
    return ResidualNormGrads(*_call("residual_norm_bwd", stream, dR, dN, R, Y, w_post, gate, alpha, w_pre, eps))


def grad_norm(grads, stream=None):
    """sqrt of the sum of all elements' squares over a list of tensors (float32 or
    bfloat16), a float32 tensor without dimensions; nothing waits for the device."""
    return _call("grad_norm", stream, grads)


def clip_grads(grads, norm, max_norm, out=None, stream=None):
    """The gradients times min(1, max_norm / norm), norm as grad_norm returns it: in
    place, or into the tensors `out`, of the same shapes (float32 or bfloat16)."""
    return _call("clip_grads", stream, grads, norm, max_norm, out)
