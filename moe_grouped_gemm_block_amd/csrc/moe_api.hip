// Host side of the mixture-of-experts operators around the FP8 products:
// argument checks (before any HIP call), launch shapes, and the kernels.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "dg.h"
#include "moe.hpp"
#include "swiglu.hpp"
#include "wgrad.hpp"

namespace dg {

#define DG_MOE_KERNEL(NAME, THREADS, ARGS, ...) \
  __global__ __launch_bounds__(THREADS) void NAME(ARGS p) { __VA_ARGS__(p); }
DG_MOE_KERNEL(dg_moe_sort_count_i32, kSortThreads, SortArgs, sort_count_body<int32_t>)
DG_MOE_KERNEL(dg_moe_sort_count_i64, kSortThreads, SortArgs, sort_count_body<int64_t>)
DG_MOE_KERNEL(dg_moe_sort_place_i32, kSortThreads, SortArgs, sort_place_body<int32_t, false>)
DG_MOE_KERNEL(dg_moe_sort_place_i64, kSortThreads, SortArgs, sort_place_body<int64_t, false>)
DG_MOE_KERNEL(dg_moe_sort_one_i32, kSortThreads, SortArgs, sort_place_body<int32_t, true>)
DG_MOE_KERNEL(dg_moe_sort_one_i64, kSortThreads, SortArgs, sort_place_body<int64_t, true>)
DG_MOE_KERNEL(dg_moe_permute_b2, 256, PermuteArgs, permute_body<2, true>)
DG_MOE_KERNEL(dg_moe_permute_b2_any, 256, PermuteArgs, permute_body<2, false>)
DG_MOE_KERNEL(dg_moe_permute_b4, 256, PermuteArgs, permute_body<4, true>)
DG_MOE_KERNEL(dg_moe_permute_b4_any, 256, PermuteArgs, permute_body<4, false>)
DG_MOE_KERNEL(dg_moe_permute_fp8_bf16_amax, 256, PermuteArgs, permute_fp8_body<true, false>)
DG_MOE_KERNEL(dg_moe_permute_fp8_bf16_pow2, 256, PermuteArgs, permute_fp8_body<true, true>)
DG_MOE_KERNEL(dg_moe_permute_fp8_f32_amax, 256, PermuteArgs, permute_fp8_body<false, false>)
DG_MOE_KERNEL(dg_moe_permute_fp8_f32_pow2, 256, PermuteArgs, permute_fp8_body<false, true>)
DG_MOE_KERNEL(dg_moe_combine_bf16, 256, CombineArgs, combine_body<true, 8>)
DG_MOE_KERNEL(dg_moe_combine_bf16_any, 256, CombineArgs, combine_body<true, 1>)
DG_MOE_KERNEL(dg_moe_combine_f32, 256, CombineArgs, combine_body<false, 4>)
DG_MOE_KERNEL(dg_moe_combine_f32_any, 256, CombineArgs, combine_body<false, 1>)
DG_MOE_KERNEL(dg_moe_combine_bwd_bf16, 256, CombineBwdArgs, combine_bwd_body<true, 8>)
DG_MOE_KERNEL(dg_moe_combine_bwd_bf16_any, 256, CombineBwdArgs, combine_bwd_body<true, 1>)
DG_MOE_KERNEL(dg_moe_combine_bwd_f32, 256, CombineBwdArgs, combine_bwd_body<false, 4>)
DG_MOE_KERNEL(dg_moe_combine_bwd_f32_any, 256, CombineBwdArgs, combine_bwd_body<false, 1>)
DG_MOE_KERNEL(dg_swiglu_fp8_bf16, 256, SwigluArgs, swiglu_body<true, true>)
DG_MOE_KERNEL(dg_swiglu_fp8_f32, 256, SwigluArgs, swiglu_body<false, true>)
DG_MOE_KERNEL(dg_swiglu_fp8_bf16_nockpt, 256, SwigluArgs, swiglu_body<true, false>)
DG_MOE_KERNEL(dg_swiglu_fp8_f32_nockpt, 256, SwigluArgs, swiglu_body<false, false>)
DG_MOE_KERNEL(dg_swiglu_fp8_bwd_bf16, 256, SwigluBwdArgs, swiglu_bwd_body<true>)
DG_MOE_KERNEL(dg_swiglu_fp8_bwd_f32, 256, SwigluBwdArgs, swiglu_bwd_body<false>)
#undef DG_MOE_KERNEL

}  // namespace dg

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// a row's bytes stay below 2^24, its pieces and blocks are counted in 32 bits
constexpr int64_t kMaxWidth = int64_t(1) << 22;
// slots are counted in 32 bits, a chunk past the last one included
constexpr int64_t kMaxSlots = int64_t(1) << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// a pointer that has to be there, aligned
bool bad(const void* p, uintptr_t a) { return p == nullptr || !aligned(p, a); }
bool valid_type(int t) { return t == DG_IN_F32 || t == DG_IN_BF16; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kGridX = int64_t(1) << dg::kGridBits;   // workgroups of a grid's row

template <typename Args>
int launch(void (*kernel)(Args), Args& a, int64_t blocks, int threads, hipStream_t stream) {
  if (blocks <= 0) return DG_OK;
  if (blocks > INT32_MAX) return DG_ERR_UNSUPPORTED;
  void* kargs[] = {&a};
  const dim3 grid(unsigned(std::min(blocks, kGridX)), unsigned(ceil_div(blocks, kGridX)));
  const hipError_t err =
      hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(unsigned(threads)), kargs, 0, stream);
  return err == hipSuccess ? DG_OK : DG_ERR_LAUNCH;
}

// Tokens, choices and width of the sorted matrix's operators.
int check_tokens(int64_t T, int top_k, int64_t M, int64_t H) {
  if (T < 0 || top_k < 1 || M < 0 || H < 0 || T > kMaxDim || M > kMaxDim || H > kMaxDim) return DG_ERR_INVALID_ARG;
  if (T * top_k > kMaxDim) return DG_ERR_INVALID_ARG;
  if (T * top_k > kMaxSlots || H > kMaxWidth) return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

// Slots and experts of the sort.
int check_sort(int64_t T, int top_k, int num_groups) {
  if (num_groups < 1) return DG_ERR_INVALID_ARG;
  const int st = check_tokens(T, top_k, 0, 0);
  if (st != DG_OK) return st;
  return num_groups > dg::kSortMaxGroups ? DG_ERR_UNSUPPORTED : DG_OK;
}

// Slots that one workgroup of the counting sort takes.
int64_t sort_chunk(int64_t slots) {
  if (slots <= dg::kSortSingle) return ceil_div(std::max<int64_t>(slots, 1), dg::kSortThreads) * dg::kSortThreads;
  // at most 128 chunks: every workgroup reads the counts of all
  return std::max<int64_t>(2048, ceil_div(ceil_div(slots, 128), dg::kSortThreads) * dg::kSortThreads);
}

int64_t rows_of(int64_t T, int top_k, int G, int align) {
  const int64_t slots = T * top_k;
  return (slots + int64_t(align - 1) * std::min<int64_t>(G, slots)) / align * align;
}

// Workgroups of four waves, sixteen rows each, that look for padding rows.
int64_t padding_blocks(int64_t M) { return ceil_div(M, 64); }

}  // namespace

extern "C" {

int64_t dg_moe_rows(int64_t T, int top_k, int num_groups, int align) {
  if (align != 1 && align != 128) return DG_ERR_INVALID_ARG;
  const int st = check_sort(T, top_k, num_groups);
  if (st != DG_OK) return st;
  return rows_of(T, top_k, num_groups, align);
}

int64_t dg_moe_sort_workspace(int64_t T, int top_k, int num_groups) {
  const int st = check_sort(T, top_k, num_groups);
  if (st != DG_OK) return st;
  const int64_t slots = T * top_k;
  return slots <= dg::kSortSingle ? 0 : 4 * ceil_div(slots, sort_chunk(slots)) * num_groups;
}

int dg_moe_sort(const void* ids, int ids_dtype, int64_t T, int top_k, int num_groups, int align, int64_t M_total,
                int32_t* group_offsets, int32_t* group_counts, int32_t* row_slot, int32_t* slot_row, void* workspace,
                hipStream_t stream) {
  if (ids_dtype != DG_IDX_I32 && ids_dtype != DG_IDX_I64) return DG_ERR_INVALID_ARG;
  if (align != 1 && align != 128) return DG_ERR_INVALID_ARG;
  if (M_total < 0 || M_total > kMaxDim) return DG_ERR_INVALID_ARG;
  const int st = check_sort(T, top_k, num_groups);
  if (st != DG_OK) return st;
  const int64_t slots = T * top_k;
  if (M_total < rows_of(T, top_k, num_groups, align) || M_total % align != 0) return DG_ERR_INVALID_ARG;
  if (bad(group_offsets, 4) || bad(group_counts, 4)) return DG_ERR_INVALID_ARG;
  if (M_total > 0 && bad(row_slot, 4)) return DG_ERR_INVALID_ARG;
  if (slots > 0 && (bad(ids, ids_dtype == DG_IDX_I64 ? 8 : 4) || bad(slot_row, 4))) return DG_ERR_INVALID_ARG;
  const int64_t chunk = sort_chunk(slots);
  const int64_t nb = std::max<int64_t>(1, ceil_div(slots, chunk));
  const bool single = slots <= dg::kSortSingle;
  if (!single && bad(workspace, 4)) return DG_ERR_INVALID_ARG;
  dg::SortArgs a{ids, int(slots), num_groups, align, int(M_total), int(chunk), int(nb), group_offsets, group_counts,
                 row_slot, slot_row, static_cast<int32_t*>(workspace)};
  const bool wide = ids_dtype == DG_IDX_I64;
  if (single) return launch(wide ? dg::dg_moe_sort_one_i64 : dg::dg_moe_sort_one_i32, a, 1, dg::kSortThreads, stream);
  const int st1 = launch(wide ? dg::dg_moe_sort_count_i64 : dg::dg_moe_sort_count_i32, a, nb, dg::kSortThreads, stream);
  if (st1 != DG_OK) return st1;
  return launch(wide ? dg::dg_moe_sort_place_i64 : dg::dg_moe_sort_place_i32, a, nb, dg::kSortThreads, stream);
}

int dg_moe_permute(const void* X, int dtype, void* Y, const int32_t* slot_row, const int32_t* row_slot, int64_t T,
                   int top_k, int64_t M_total, int64_t H, hipStream_t stream) {
  if (!valid_type(dtype)) return DG_ERR_INVALID_ARG;
  const int st = check_tokens(T, top_k, M_total, H);
  if (st != DG_OK) return st;
  if (M_total == 0 || H == 0) return DG_OK;
  if (bad(Y, 16) || bad(row_slot, 4)) return DG_ERR_INVALID_ARG;
  if (T > 0 && (bad(X, 16) || bad(slot_row, 4))) return DG_ERR_INVALID_ARG;
  const bool b2 = dtype == DG_IN_BF16;
  const int elem = b2 ? 2 : 4;
  const bool wide = H * elem % 16 == 0;
  const int64_t main = ceil_div(T * (wide ? H * elem / 16 : H), 256);
  if (main + padding_blocks(M_total) > INT32_MAX) return DG_ERR_UNSUPPORTED;
  dg::PermuteArgs a{X, Y, nullptr, slot_row, row_slot, int(T), top_k, int(M_total), int(H), 0, int(main)};
  return launch(b2 ? (wide ? dg::dg_moe_permute_b2 : dg::dg_moe_permute_b2_any)
                   : (wide ? dg::dg_moe_permute_b4 : dg::dg_moe_permute_b4_any),
                a, main + padding_blocks(M_total), 256, stream);
}

int dg_moe_permute_fp8(const void* X, int in_dtype, void* Q, float* S, int scale_mode, const int32_t* slot_row,
                       const int32_t* row_slot, int64_t T, int top_k, int64_t M_total, int64_t H, hipStream_t stream) {
  if (!valid_type(in_dtype)) return DG_ERR_INVALID_ARG;
  if (scale_mode != DG_SCALE_AMAX && scale_mode != DG_SCALE_POW2) return DG_ERR_INVALID_ARG;
  const int st = check_tokens(T, top_k, M_total, H);
  if (st != DG_OK) return st;
  if (M_total == 0 || H == 0) return DG_OK;
  if (bad(Q, 16) || bad(S, 4) || bad(row_slot, 4)) return DG_ERR_INVALID_ARG;
  if (T > 0 && (bad(X, 16) || bad(slot_row, 4))) return DG_ERR_INVALID_ARG;
  if (H % 16 != 0) return DG_ERR_UNSUPPORTED;
  const int64_t Kb = ceil_div(H, 128);
  const int64_t main = ceil_div(T * Kb, 32);
  if (main + padding_blocks(M_total) > INT32_MAX) return DG_ERR_UNSUPPORTED;
  dg::PermuteArgs a{X, Q, S, slot_row, row_slot, int(T), top_k, int(M_total), int(H), int(Kb), int(main)};
  const bool bf16 = in_dtype == DG_IN_BF16, pow2 = scale_mode == DG_SCALE_POW2;
  return launch(bf16 ? (pow2 ? dg::dg_moe_permute_fp8_bf16_pow2 : dg::dg_moe_permute_fp8_bf16_amax)
                     : (pow2 ? dg::dg_moe_permute_fp8_f32_pow2 : dg::dg_moe_permute_fp8_f32_amax),
                a, main + padding_blocks(M_total), 256, stream);
}

int dg_moe_combine(const void* Y, int dtype, const float* weights, const int32_t* slot_row, void* out, int64_t T,
                   int top_k, int64_t M_total, int64_t H, hipStream_t stream) {
  if (!valid_type(dtype)) return DG_ERR_INVALID_ARG;
  const int st = check_tokens(T, top_k, M_total, H);
  if (st != DG_OK) return st;
  if (T == 0 || H == 0) return DG_OK;
  if (bad(out, 16) || bad(slot_row, 4) || !aligned(weights, 4)) return DG_ERR_INVALID_ARG;
  if (M_total > 0 && bad(Y, 16)) return DG_ERR_INVALID_ARG;
  const bool bf16 = dtype == DG_IN_BF16;
  const int vec = bf16 ? 8 : 4;
  const bool wide = H % vec == 0;
  dg::CombineArgs a{Y, weights, slot_row, out, int(T), top_k, int(M_total), int(H)};
  return launch(bf16 ? (wide ? dg::dg_moe_combine_bf16 : dg::dg_moe_combine_bf16_any)
                     : (wide ? dg::dg_moe_combine_f32 : dg::dg_moe_combine_f32_any),
                a, ceil_div(T * (wide ? H / vec : H), 256), 256, stream);
}

int dg_moe_combine_bwd(const void* dOut, const void* Y, int dtype, const float* weights, const int32_t* slot_row,
                       const int32_t* row_slot, void* dY, float* dweights, int64_t T, int top_k, int64_t M_total,
                       int64_t H, hipStream_t stream) {
  if (!valid_type(dtype)) return DG_ERR_INVALID_ARG;
  const int st = check_tokens(T, top_k, M_total, H);
  if (st != DG_OK) return st;
  if (T > 0 && (bad(weights, 4) || bad(slot_row, 4) || bad(dweights, 4) || (H > 0 && bad(dOut, 16))))
    return DG_ERR_INVALID_ARG;
  if (M_total > 0 && (bad(row_slot, 4) || (H > 0 && (bad(Y, 16) || bad(dY, 16))))) return DG_ERR_INVALID_ARG;
  const bool bf16 = dtype == DG_IN_BF16;
  const bool wide = H % (bf16 ? 8 : 4) == 0;
  if (T + padding_blocks(M_total) > INT32_MAX) return DG_ERR_UNSUPPORTED;
  dg::CombineBwdArgs a{dOut, Y, weights, slot_row, row_slot, dY, dweights, int(T), top_k, int(M_total), int(H)};
  return launch(bf16 ? (wide ? dg::dg_moe_combine_bwd_bf16 : dg::dg_moe_combine_bwd_bf16_any)
                     : (wide ? dg::dg_moe_combine_bwd_f32 : dg::dg_moe_combine_bwd_f32_any),
                a, T + padding_blocks(M_total), 256, stream);
}

int dg_swiglu_fp8(const void* H, int in_dtype, void* A, float* sA, void* Hq, float* sH, int64_t M, int64_t I,
                  hipStream_t stream) {
  if (!valid_type(in_dtype)) return DG_ERR_INVALID_ARG;
  if (M < 0 || I < 0 || M > kMaxDim || I > kMaxDim) return DG_ERR_INVALID_ARG;
  if ((Hq == nullptr) != (sH == nullptr)) return DG_ERR_INVALID_ARG;
  if (M == 0 || I == 0) return DG_OK;
  if (bad(H, 16) || bad(A, 16) || bad(sA, 4) || !aligned(Hq, 16) || !aligned(sH, 4)) return DG_ERR_INVALID_ARG;
  if (I % 16 != 0 || I > kMaxWidth) return DG_ERR_UNSUPPORTED;
  const int64_t Ib = ceil_div(I, 128);
  dg::SwigluArgs a{H, static_cast<uint8_t*>(A), sA, static_cast<uint8_t*>(Hq), sH, int(M), int(I), int(Ib)};
  const bool bf16 = in_dtype == DG_IN_BF16;
  return launch(Hq ? (bf16 ? dg::dg_swiglu_fp8_bf16 : dg::dg_swiglu_fp8_f32)
                   : (bf16 ? dg::dg_swiglu_fp8_bf16_nockpt : dg::dg_swiglu_fp8_f32_nockpt),
                a, ceil_div(M * Ib, 32), 256, stream);
}

int dg_swiglu_fp8_bwd(const void* dA, int dtype, const void* Hq, const float* sH, void* dH, int64_t M, int64_t I,
                      hipStream_t stream) {
  if (!valid_type(dtype)) return DG_ERR_INVALID_ARG;
  if (M < 0 || I < 0 || M > kMaxDim || I > kMaxDim) return DG_ERR_INVALID_ARG;
  if (M == 0 || I == 0) return DG_OK;
  if (bad(dA, 16) || bad(Hq, 16) || bad(sH, 4) || bad(dH, 16)) return DG_ERR_INVALID_ARG;
  if (I % 16 != 0 || I > kMaxWidth) return DG_ERR_UNSUPPORTED;
  dg::SwigluBwdArgs a{dA, static_cast<const uint8_t*>(Hq), sH, dH, int(M), int(I), int(ceil_div(I, 128))};
  return launch(dtype == DG_IN_BF16 ? dg::dg_swiglu_fp8_bwd_bf16 : dg::dg_swiglu_fp8_bwd_f32, a,
                ceil_div(M * (I / 8), 256), 256, stream);
}

int dg_grouped_wgrad_fp8(const void* dY, const void* X, const float* sX, const int32_t* group_offsets,
                         const int32_t* group_counts, int num_groups, int64_t M_total, int64_t N, int64_t K, void* dW,
                         int out_dtype, int accumulate, hipStream_t stream) {
  if (out_dtype != DG_OUT_F32 && out_dtype != DG_OUT_BF16) return DG_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return DG_ERR_INVALID_ARG;
  if (num_groups < 1 || M_total < 0 || N < 0 || K < 0 || M_total > kMaxDim || N > kMaxDim || K > kMaxDim)
    return DG_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return DG_OK;
  if (bad(dW, 16) || bad(group_offsets, 4) || !aligned(group_counts, 4)) return DG_ERR_INVALID_ARG;
  if (M_total > 0 && (bad(dY, 16) || bad(X, 16) || bad(sX, 4))) return DG_ERR_INVALID_ARG;
  // rows of dY and X start 16-byte aligned
  if (N % 8 != 0 || K % 16 != 0 || N > kMaxWidth || K > kMaxWidth) return DG_ERR_UNSUPPORTED;
  dg::WgradArgs a{static_cast<const uint16_t*>(dY), static_cast<const uint8_t*>(X), sX, group_offsets, group_counts,
                  dW, num_groups, int(M_total), int(N), int(K), int(ceil_div(K, 128)), 0, 0, 0, accumulate};
  const bool bf16 = out_dtype == DG_OUT_BF16;
  // 256 x 128 tiles from more than one per CU (256) on, 128 x 128 below (FP32,
  // 256 x 128 against 128 x 128: 64 tiles of 1024 rows 23.9 / 17.7 us, 256 of 256
  // rows 15.2 / 13.2, 320 of 1024 rows 36.0 / 38.7, 384 of 256 rows 19.6 / 19.6, 512
  // of 512 rows 28.6 / 33.2)
  const bool big = num_groups * ceil_div(N, 256) * ceil_div(K, 128) > 256;
  a.n_tiles = int(ceil_div(N, big ? 256 : 128));
  a.k_tiles = int(ceil_div(K, 128));
  const int64_t tiles = int64_t(a.n_tiles) * a.k_tiles;
  // (fewer tiles would leave XCDs without work: the last eighth may be short)
  a.per_xcd = tiles >= 64 ? int(ceil_div(tiles, 8)) : 0;
  const int64_t blocks = num_groups * (a.per_xcd ? 8 * int64_t(a.per_xcd) : tiles);
  if (blocks > kGridX) return DG_ERR_UNSUPPORTED;   // one row of a grid
  return launch(big ? (bf16 ? dg::dg_wgrad256_bf16 : dg::dg_wgrad256_f32)
                    : (bf16 ? dg::dg_wgrad128_bf16 : dg::dg_wgrad128_f32),
                a, blocks, 256, stream);
}

}  // extern "C"
