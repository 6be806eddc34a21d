// Host side of the operators that make the mixture-of-experts layer a block of a
// model: the router, the norms around the block, and gradient clipping.  Argument
// checks (before any HIP call), launch shapes, and the kernels.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>
#include <type_traits>

#include "clip.hpp"
#include "dg.h"
#include "host.hpp"
#include "norm.hpp"
#include "route.hpp"

namespace dg {

#define DG_BLOCK_KERNEL(NAME, THREADS, ARGS, ...) \
  __global__ __launch_bounds__(THREADS) void NAME(ARGS p) { __VA_ARGS__(p); }
#define DG_ROUTE_KERNELS(T, BF16)                                                                      \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_16x4, kRouteThreads, RouteArgs, route_body<BF16, 16, 4, false>)          \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_16x16, kRouteThreads, RouteArgs, route_body<BF16, 16, 16, false>)        \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_64x4, kRouteThreads, RouteArgs, route_body<BF16, 64, 4, false>)          \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_64x16, kRouteThreads, RouteArgs, route_body<BF16, 64, 16, false>)        \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_16x4_bias, kRouteThreads, RouteArgs, route_body<BF16, 16, 4, true>)      \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_16x16_bias, kRouteThreads, RouteArgs, route_body<BF16, 16, 16, true>)    \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_64x4_bias, kRouteThreads, RouteArgs, route_body<BF16, 64, 4, true>)      \
  DG_BLOCK_KERNEL(dg_moe_route_##T##_64x16_bias, kRouteThreads, RouteArgs, route_body<BF16, 64, 16, true>)    \
  DG_BLOCK_KERNEL(dg_moe_route_bwd_##T##_16x4, kRouteBwdThreads, RouteBwdArgs, route_bwd_body<BF16, 16, 4>)   \
  DG_BLOCK_KERNEL(dg_moe_route_bwd_##T##_16x16, kRouteBwdThreads, RouteBwdArgs, route_bwd_body<BF16, 16, 16>) \
  DG_BLOCK_KERNEL(dg_moe_route_bwd_##T##_64x4, kRouteBwdThreads, RouteBwdArgs, route_bwd_body<BF16, 64, 4>)   \
  DG_BLOCK_KERNEL(dg_moe_route_bwd_##T##_64x16, kRouteBwdThreads, RouteBwdArgs, route_bwd_body<BF16, 64, 16>)
DG_ROUTE_KERNELS(bf16, true)
DG_ROUTE_KERNELS(f32, false)
DG_BLOCK_KERNEL(dg_moe_route_finish, kFinishExperts * kFinishParts, RouteArgs, route_finish_body)
DG_BLOCK_KERNEL(dg_moe_route_finish_one, kFinishExperts * kFinishParts, RouteArgs, route_finish_one_body)
#undef DG_ROUTE_KERNELS

// (templates: stream and value types, codes, whole rows, wide rows)
template <bool RB, bool YB, int CODES, bool WHOLE, bool WIDE>
DG_BLOCK_KERNEL(dg_residual_norm_kernel, WIDE ? kNormWideThreads : kNormMaxThreads, NormArgs,
                norm_body<RB, YB, CODES, WHOLE, WIDE>)
template <bool RB, bool YB, bool WHOLE, bool WIDE>
DG_BLOCK_KERNEL(dg_residual_norm_bwd_kernel, WIDE || (!WHOLE && !(RB && YB)) ? kNormWideThreads : kNormMaxThreads,
                NormBwdArgs, norm_bwd_body<RB, YB, WHOLE, WIDE>)
DG_BLOCK_KERNEL(dg_residual_norm_columns, 1024, NormColumnsArgs, norm_columns_body)

DG_BLOCK_KERNEL(dg_grad_squares, kClipThreads, ClipBatch, clip_squares_body)
DG_BLOCK_KERNEL(dg_grad_norm_sum, kClipNormThreads, ClipNormArgs, clip_norm_body)
DG_BLOCK_KERNEL(dg_grad_norm_few, kClipNormThreads, ClipBatch, clip_norm_few_body)
DG_BLOCK_KERNEL(dg_clip_scale, kClipThreads, ClipBatch, clip_scale_body)
#undef DG_BLOCK_KERNEL

}  // namespace dg

namespace {

using namespace dg_host;

int elem(int dtype) { return dtype == DG_IN_BF16 ? 2 : 4; }

// ---- router ------------------------------------------------------------------------

int check_route(int64_t T, int64_t E, int top_k) {
  if (T < 0 || E < 1 || top_k < 1 || T > kMaxDim || E > kMaxDim || top_k > E || T * top_k > kMaxDim)
    return DG_ERR_INVALID_ARG;
  if (E > dg::kRouteMaxExperts || top_k > 64 || T * top_k > kMaxSlots) return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

// Lanes and logits per lane: a row of 16 lanes holds up to 256 experts and 16 choices.
// More than 64 experts of few tokens go over a whole wave each, which ends sooner, many
// over a row, which takes fewer instructions a token (256 experts, 8 choices, biased
// sigmoid with the load, row / wave: 256 tokens 14.3 / 10.4 us, 4096 15.8 / 14.9, 8192 17.4
// / 18.7, 16384 19.6 / 26.5; gradient 4096 5.1 / 4.9, 8192 7.1 / 7.9).
int route_lanes(int64_t T, int64_t E, int top_k) {
  return E <= 256 && top_k <= 16 && (E <= 64 || T > 4096) ? 16 : 64;
}
int route_variant(int64_t T, int64_t E, int top_k) {
  if (route_lanes(T, E, top_k) == 16) return E <= 64 ? 0 : 1;
  return E <= 256 ? 2 : 3;
}

// Workgroups.  With the load a single one takes few tokens, which saves the second launch
// (64 experts, a row of lanes a token: 128 tokens in two turns 6.4 us, by two launches 9.6;
// a wave a token, 256 experts: 16 tokens in one turn 5.9 us, 64 in four 14.9, by two
// launches 9.5).
int64_t route_blocks(int64_t T, int64_t E, int top_k, bool balance) {
  const int lanes = route_lanes(T, E, top_k);
  if (balance && T <= (lanes == 16 ? 128 : 16)) return 1;
  return std::min<int64_t>(std::max<int64_t>(1, ceil_div(T, dg::kRouteThreads / lanes)),
                           balance ? dg::kRouteMaxBlocks : 65536);
}

// Alignment of logits: of a vector of four where rows are of whole ones.
int route_align(int dtype, int64_t E) { return (E % 4 == 0 ? 4 : 1) * elem(dtype); }

bool valid_scores(int score, int renormalise, float scale) {
  return (score == DG_SCORE_SOFTMAX || score == DG_SCORE_SIGMOID) && (renormalise == 0 || renormalise == 1) &&
         isfinite(scale);
}

// ---- norms -------------------------------------------------------------------------

// Alignment of a matrix or of weights: of 16 bytes where rows are of whole vectors, others
// start at any element.
int norm_align(int dtype, int64_t H) { return H % 8 == 0 ? 16 : elem(dtype); }

// Threads of a row that fits `most` threads' registers, or of a wider one.
int norm_threads(int64_t H, int64_t most = dg::kNormMaxThreads) {
  const int64_t threads = ceil_div(ceil_div(H, dg::kNormColumns), 64) * 64;
  return int(threads <= most ? threads : dg::kNormWideThreads);
}
bool norm_wide(int64_t H, int64_t most = dg::kNormMaxThreads) { return H > dg::kNormColumns * most; }

// The backward pass of FP32 rows that start at any element takes more registers.
int64_t norm_bwd_most(int64_t H, bool bf16) { return H % 8 == 0 || bf16 ? dg::kNormMaxThreads : dg::kNormWideThreads; }

// Rows that a workgroup of the backward pass takes at a time: as many as 8 waves hold.
// (Fewer waves a workgroup would leave CUs without work to hide latency behind, more
// workgroups would write more partial sums: 8192 rows of 512 28 us one at a time, 15 so.)
int norm_bwd_groups(int64_t H) { return std::max(1, dg::kNormGroupThreads / norm_threads(H)); }
// Where larger workgroups, up to `most` threads, take all rows in one turn, one on a CU:
// fewer partial sums and none of the CUs with two turns (1009 rows of 1408, FP32 stream, 12.9
// -> 12.2 us; 600 of 2048 12.9 -> 11.5, 512 of 4096 17.3 -> 14.8, 4000 of 512 11.7 -> 11.3).
int norm_bwd_groups(int64_t T, int64_t H, int64_t most) {
  const int groups = norm_bwd_groups(H);
  const int64_t one_turn = ceil_div(T, 256);
  return norm_wide(H, most) || one_turn * norm_threads(H) > most ? groups : std::max(groups, int(one_turn));
}

// (at most: larger workgroups are fewer)
int64_t norm_bwd_blocks(int64_t T, int64_t H) {
  // (partial sums of 16 MB at most for wide rows)
  const int64_t most = norm_wide(H) ? std::max<int64_t>(1, (int64_t(1) << 22) / H) : 512;
  return std::min(ceil_div(T, norm_bwd_groups(H)), std::min<int64_t>(most, 512));
}

constexpr int64_t kNormAloneTurns = 2;

int check_norm(int r_dtype, int dtype, const void* Y, const float* w_post, const float* gate, int gate_kind,
               float alpha, const float* w_pre, float eps, int64_t T, int64_t H) {
  if (!valid_type(r_dtype) || !valid_type(dtype)) return DG_ERR_INVALID_ARG;
  if (gate_kind != DG_GATE_NONE && gate_kind != DG_GATE_CHANNEL && gate_kind != DG_GATE_TOKEN) return DG_ERR_INVALID_ARG;
  if (!isfinite(alpha) || !isfinite(eps) || !(eps > 0.f)) return DG_ERR_INVALID_ARG;
  if (T < 0 || H < 1 || T > kMaxDim || H > kMaxDim) return DG_ERR_INVALID_ARG;
  // (what has no rows may have no address)
  if (T > 0 && Y == nullptr && (w_post || gate || gate_kind != DG_GATE_NONE || !w_pre)) return DG_ERR_INVALID_ARG;
  if ((gate == nullptr) != (gate_kind == DG_GATE_NONE) && !(T == 0 && gate_kind == DG_GATE_TOKEN)) return DG_ERR_INVALID_ARG;
  const int weights = norm_align(DG_IN_F32, H);
  if (!aligned(Y, norm_align(dtype, H)) || !aligned(w_post, weights) ||
      !aligned(gate, gate_kind == DG_GATE_TOKEN ? 4 : weights) || !aligned(w_pre, weights))
    return DG_ERR_INVALID_ARG;
  return DG_OK;
}

template <bool RB, bool YB, int CODES>
void (*norm_kernel(bool whole, bool wide))(dg::NormArgs) {
  if constexpr (CODES != dg::kCodesNone) {
    return wide ? dg::dg_residual_norm_kernel<RB, YB, CODES, true, true>
                : dg::dg_residual_norm_kernel<RB, YB, CODES, true, false>;
  } else {
    return whole ? (wide ? dg::dg_residual_norm_kernel<RB, YB, CODES, true, true>
                         : dg::dg_residual_norm_kernel<RB, YB, CODES, true, false>)
                 : (wide ? dg::dg_residual_norm_kernel<RB, YB, CODES, false, true>
                         : dg::dg_residual_norm_kernel<RB, YB, CODES, false, false>);
  }
}

template <bool RB, bool YB>
void (*norm_kernel(int codes, bool whole, bool wide))(dg::NormArgs) {
  return codes == dg::kCodesNone   ? norm_kernel<RB, YB, dg::kCodesNone>(whole, wide)
         : codes == dg::kCodesPow2 ? norm_kernel<RB, YB, dg::kCodesPow2>(whole, wide)
                                   : norm_kernel<RB, YB, dg::kCodesAmax>(whole, wide);
}

template <bool RB, bool YB>
void (*norm_bwd_kernel(bool whole, bool wide))(dg::NormBwdArgs) {
  return whole ? (wide ? dg::dg_residual_norm_bwd_kernel<RB, YB, true, true>
                       : dg::dg_residual_norm_bwd_kernel<RB, YB, true, false>)
               : (wide ? dg::dg_residual_norm_bwd_kernel<RB, YB, false, true>
                       : dg::dg_residual_norm_bwd_kernel<RB, YB, false, false>);
}

// ---- clipping ------------------------------------------------------------------------

// Sizes and types of a list of tensors; its chunks, or a negative status.
int64_t clip_chunks(const int64_t* sizes, const int* dtypes, int count) {
  if (count < 0 || (count > 0 && (sizes == nullptr || dtypes == nullptr))) return DG_ERR_INVALID_ARG;
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > (int64_t(1) << 45) || !valid_type(dtypes[i])) return DG_ERR_INVALID_ARG;
    chunks += ceil_div(sizes[i], dg::kClipChunk);
    if (chunks > kMaxDim) return DG_ERR_UNSUPPORTED;
  }
  return chunks;
}

// Whether what the outputs' addresses cover is written once, and read by no other
// tensor's and not by the norm's: ranges in order of their addresses, grads[i] itself
// counting for outs[i].  -1: no memory to sort them in.
int clip_disjoint(const void* const* grads, const int64_t* sizes, const int* dtypes, int count, void* const* outs,
                  const int* out_dtypes, const float* norm) {
  struct Range {
    uintptr_t begin, end;
    bool out;
  };
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * size_t(count) + 1]);
  if (!r) return -1;
  size_t n = 0;
  bool sorted = true;
  auto add = [&](const void* p, int64_t bytes, bool out) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    r[n] = Range{a, a + uintptr_t(bytes), out};
    sorted = sorted && (n == 0 || r[n - 1].begin <= a);
    ++n;
  };
  for (int i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    if (grads[i] != outs[i]) add(grads[i], sizes[i] * elem(dtypes[i]), false);
    add(outs[i], sizes[i] * elem(out_dtypes[i]), true);
  }
  add(norm, sizeof(float), false);
  if (!sorted) std::sort(r.get(), r.get() + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t any = 0, out = 0;                       // ends of the ranges so far, and of the outputs among them
  for (size_t i = 0; i < n; ++i) {
    if (r[i].begin < (r[i].out ? any : out)) return 0;
    any = std::max(any, r[i].end);
    if (r[i].out) out = std::max(out, r[i].end);
  }
  return 1;
}

// Whether one workgroup takes the norm, in one launch instead of two (norm and clipping of
// the small tensors of a layer 9.6 us, 13.3 with three launches; at kClipFew elements the
// norm takes about 5 us either way).
bool clip_few(const int64_t* sizes, int count) {
  int64_t n = 0;
  int tensors = 0;
  for (int i = 0; i < count; ++i) {
    n += sizes[i];
    tensors += sizes[i] > 0;
    if (n > dg::kClipFew || tensors > dg::kClipTensors) return false;
  }
  return true;
}

// The launches of a kernel over a list, up to kClipTensors tensors that are not empty
// each; `fill` completes a tensor's entry.
template <typename F>
int clip_launches(void (*kernel)(dg::ClipBatch), dg::ClipBatch& b, const void* const* grads, const int64_t* sizes,
                  const int* dtypes, int count, hipStream_t stream, F fill, bool few = false) {
  b.count = b.chunks = 0;
  for (int i = 0; i <= count; ++i) {
    const int64_t chunks = i < count ? ceil_div(sizes[i], dg::kClipChunk) : 0;
    if (b.count == dg::kClipTensors || (i == count && b.count > 0)) {
      const int st = launch(kernel, b, few ? 1 : b.chunks, few ? dg::kClipNormThreads : dg::kClipThreads, stream);
      if (st != DG_OK) return st;
      if (b.part) b.part += b.chunks;
      b.count = b.chunks = 0;
    }
    if (chunks == 0) continue;
    dg::ClipTensor& t = b.t[b.count++];
    t = dg::ClipTensor{grads[i], nullptr, sizes[i], b.chunks, uint8_t(dtypes[i] == DG_IN_BF16), 0,
                       uint8_t(aligned(grads[i], 16)), 0};
    fill(t, i);
    b.chunks += int(chunks);
  }
  return DG_OK;
}

}  // namespace

extern "C" {

int64_t dg_moe_route_workspace(int64_t T, int64_t E, int top_k) {
  const int st = check_route(T, E, top_k);
  if (st != DG_OK) return st;
  const int64_t nb = route_blocks(T, E, top_k, true);
  return nb > 1 ? nb * (8 * E + 4) + 8 * E + 4 : 0;
}

int dg_moe_route(const void* logits, int dtype, const float* bias, const uint8_t* mask, int64_t T, int64_t E, int top_k,
                 int score, int renormalise, float scale, int32_t* ids, float* weights, int32_t* counts,
                 float* prob_sums, int32_t* routed, float* loss, void* workspace, hipStream_t stream) {
  if (!valid_type(dtype) || !valid_scores(score, renormalise, scale)) return DG_ERR_INVALID_ARG;
  const int st = check_route(T, E, top_k);
  if (st != DG_OK) return st;
  const bool balance = counts != nullptr;
  if ((prob_sums != nullptr) != balance || (routed != nullptr) != balance || (loss != nullptr) != balance)
    return DG_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(prob_sums, 4) || !aligned(routed, 4) || !aligned(loss, 4) || !aligned(bias, 4))
    return DG_ERR_INVALID_ARG;
  const int64_t nb = route_blocks(T, E, top_k, balance);
  if (balance && nb > 1 && bad(workspace, 8)) return DG_ERR_INVALID_ARG;
  if (T > 0 && (bad(logits, route_align(dtype, E)) || bad(ids, 4) || bad(weights, 4))) return DG_ERR_INVALID_ARG;
  if (T == 0 && !balance) return DG_OK;
  double* terms = static_cast<double*>(nb > 1 && balance ? workspace : nullptr);
  float* part = terms ? reinterpret_cast<float*>(terms + E) : nullptr;
  int32_t* ints = terms ? reinterpret_cast<int32_t*>(part + nb * E) : nullptr;
  dg::RouteArgs a{logits, bias, mask, ids, weights, counts, prob_sums, routed, loss, part, ints,
                  terms ? ints + nb * E : nullptr, terms, terms ? ints + nb * E + nb : nullptr, int(T), int(E), top_k,
                  int(nb), score == DG_SCORE_SIGMOID, renormalise, aligned(bias, 16), scale};
#define DG_ROUTE_TABLE(T)                                                                                       \
  {{dg::dg_moe_route_##T##_16x4, dg::dg_moe_route_##T##_16x16, dg::dg_moe_route_##T##_64x4,                     \
    dg::dg_moe_route_##T##_64x16},                                                                              \
   {dg::dg_moe_route_##T##_16x4_bias, dg::dg_moe_route_##T##_16x16_bias, dg::dg_moe_route_##T##_64x4_bias,      \
    dg::dg_moe_route_##T##_64x16_bias}}
  static void (*const kernels[2][2][4])(dg::RouteArgs) = {DG_ROUTE_TABLE(f32), DG_ROUTE_TABLE(bf16)};
#undef DG_ROUTE_TABLE
  const int st1 = launch(kernels[dtype == DG_IN_BF16][bias != nullptr][route_variant(T, E, top_k)], a, nb,
                         dg::kRouteThreads, stream);
  if (st1 != DG_OK || !balance || nb == 1) return st1;
  if (nb * E <= dg::kFinishOne)
    return launch(dg::dg_moe_route_finish_one, a, 1, dg::kFinishExperts * dg::kFinishParts, stream);
  return launch(dg::dg_moe_route_finish, a, ceil_div(E, dg::kFinishExperts), dg::kFinishExperts * dg::kFinishParts,
                stream);
}

int dg_moe_route_bwd(const float* dweights, const void* logits, int dtype, const int32_t* ids, const int32_t* counts,
                     const int32_t* routed, const float* dloss, int64_t T, int64_t E, int top_k, int score,
                     int renormalise, float scale, void* dlogits, hipStream_t stream) {
  if (!valid_type(dtype) || !valid_scores(score, renormalise, scale)) return DG_ERR_INVALID_ARG;
  const int st = check_route(T, E, top_k);
  if (st != DG_OK) return st;
  if ((routed != nullptr) != (counts != nullptr) || (dloss != nullptr) != (counts != nullptr)) return DG_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(routed, 4) || !aligned(dloss, 4)) return DG_ERR_INVALID_ARG;
  if (T == 0) return DG_OK;
  const int align = route_align(dtype, E);
  if (bad(dweights, 4) || bad(logits, align) || bad(ids, 4) || bad(dlogits, align)) return DG_ERR_INVALID_ARG;
  dg::RouteBwdArgs a{logits, ids, dweights, counts, routed, dloss, dlogits, int(T), int(E), top_k,
                     score == DG_SCORE_SIGMOID, renormalise, aligned(counts, 16), scale};
#define DG_ROUTE_TABLE(T)                                                                                       \
  {dg::dg_moe_route_bwd_##T##_16x4, dg::dg_moe_route_bwd_##T##_16x16, dg::dg_moe_route_bwd_##T##_64x4,          \
   dg::dg_moe_route_bwd_##T##_64x16}
  static void (*const kernels[2][4])(dg::RouteBwdArgs) = {DG_ROUTE_TABLE(f32), DG_ROUTE_TABLE(bf16)};
#undef DG_ROUTE_TABLE
  return launch(kernels[dtype == DG_IN_BF16][route_variant(T, E, top_k)], a,
                ceil_div(T, dg::kRouteBwdThreads / route_lanes(T, E, top_k)), dg::kRouteBwdThreads, stream);
}

int dg_residual_norm(const void* R, int r_dtype, const void* Y, int dtype, const float* w_post, const float* gate,
                     int gate_kind, float alpha, const float* w_pre, float eps, void* R_out, void* N, void* Q, float* S,
                     int scale_mode, int64_t T, int64_t H, hipStream_t stream) {
  const int st = check_norm(r_dtype, dtype, Y, w_post, gate, gate_kind, alpha, w_pre, eps, T, H);
  if (st != DG_OK) return st;
  if (scale_mode != DG_SCALE_AMAX && scale_mode != DG_SCALE_POW2) return DG_ERR_INVALID_ARG;
  if ((Q == nullptr) != (S == nullptr)) return DG_ERR_INVALID_ARG;
  if (T == 0) return DG_OK;
  const int of_r = norm_align(r_dtype, H), of_y = norm_align(dtype, H);
  if (bad(R, of_r) || !aligned(R_out, of_r) || !aligned(N, of_y) || !aligned(Q, 16) || !aligned(S, 4))
    return DG_ERR_INVALID_ARG;
  if ((R_out != nullptr) != (Y != nullptr) || (N != nullptr || Q != nullptr) != (w_pre != nullptr))
    return DG_ERR_INVALID_ARG;
  if (R_out && (R_out == R || R_out == Y)) return DG_ERR_INVALID_ARG;
  if (N && (N == R || N == Y)) return DG_ERR_INVALID_ARG;
  if (H > kMaxWidth || (Q && H % 16 != 0)) return DG_ERR_UNSUPPORTED;
  const bool wide = norm_wide(H), whole = H % 8 == 0;
  const int threads = norm_threads(H);
  dg::NormArgs a{R, Y, w_post, gate, w_pre, R_out, N, static_cast<uint8_t*>(Q), S, eps, 1.0 / double(H), alpha, int(T), int(H),
                 int(ceil_div(H, 128)), gate_kind};
  const int codes = !Q ? dg::kCodesNone : scale_mode == DG_SCALE_POW2 ? dg::kCodesPow2 : dg::kCodesAmax;
  const bool rb = r_dtype == DG_IN_BF16, yb = dtype == DG_IN_BF16;
  const auto kernel = rb ? (yb ? norm_kernel<true, true>(codes, whole, wide) : norm_kernel<true, false>(codes, whole, wide))
                         : (yb ? norm_kernel<false, true>(codes, whole, wide) : norm_kernel<false, false>(codes, whole, wide));
  // as many workgroups as are there at a time by their registers, three of 8 waves a CU, for
  // codes two (8192 rows of 4096: 2 a CU 48.5, 3 47.5, 4 51 us; codes 2 66, 3 70).  One of 13 to
  // 16 waves for 6145 to 8192 columns keeps up too (4096 rows of 8192 46 us, 5.8 TB/s)
  return launch(kernel, a, std::min<int64_t>(T, 256 * std::max(1, (Q ? 16 : 24) / (threads / 64))), threads, stream);
}

int64_t dg_residual_norm_bwd_workspace(int64_t T, int64_t H, int sums) {
  if (T < 0 || H < 1 || T > kMaxDim || H > kMaxDim || sums < 0 || sums > 2) return DG_ERR_INVALID_ARG;
  if (H > kMaxWidth) return DG_ERR_UNSUPPORTED;
  return 4 * norm_bwd_blocks(T, H) * H * sums;
}

int dg_residual_norm_bwd(const void* dR, const void* dN, const void* R, int r_dtype, const void* Y, int dtype,
                         const float* w_post, const float* gate, int gate_kind, float alpha, const float* w_pre,
                         float eps, void* dR_out, void* dY, float* dw_post, float* dgate, float* dw_pre, int64_t T,
                         int64_t H, void* workspace, hipStream_t stream) {
  const int st = check_norm(r_dtype, dtype, Y, w_post, gate, gate_kind, alpha, w_pre, eps, T, H);
  if (st != DG_OK) return st;
  const bool token = gate_kind == DG_GATE_TOKEN, channel = gate_kind == DG_GATE_CHANNEL;
  if (H > kMaxWidth) return DG_ERR_UNSUPPORTED;
  if ((w_pre && bad(dw_pre, 4)) || (w_post && bad(dw_post, 4)) || (channel && bad(dgate, 4))) return DG_ERR_INVALID_ARG;
  if ((!w_pre && dw_pre) || (!w_post && dw_post) || (gate_kind == DG_GATE_NONE && dgate)) return DG_ERR_INVALID_ARG;
  const bool pre = w_pre != nullptr, post = w_post != nullptr || channel;
  // few rows: one workgroup, whose sums are the gradients themselves (unless two gradients
  // come of one sum), and no second launch (4 rows of 2048 8.2 us, by two launches 9.4; 2 of
  // 4096 7.0 and 9.3)
  const bool alone = T > 0 && T <= kNormAloneTurns * norm_bwd_groups(H) && !(w_post && channel) &&
                     aligned(dw_pre, 16) && aligned(dw_post, 16) && (!channel || aligned(dgate, 16));
  const int64_t most = norm_bwd_most(H, r_dtype == DG_IN_BF16 && dtype == DG_IN_BF16);
  const int groups = norm_bwd_groups(T, H, most);
  const int64_t nb = alone ? 1 : std::min(norm_bwd_blocks(T, H), ceil_div(T, groups));
  float* part = static_cast<float*>(workspace);
  float* part_pre = !pre ? nullptr : alone ? dw_pre : part;
  float* part_post = !post ? nullptr : alone ? (w_post ? dw_post : dgate) : part + (pre ? nb * H : 0);
  if (T > 0) {
    const int of_r = norm_align(r_dtype, H), of_y = norm_align(dtype, H);
    if (bad(dR_out, of_r) || !aligned(dR, of_r) || (token && bad(dgate, 4))) return DG_ERR_INVALID_ARG;
    if (pre ? bad(R, of_r) || bad(dN, of_y) : dN != nullptr || dR == nullptr) return DG_ERR_INVALID_ARG;
    if ((dY != nullptr) != (Y != nullptr) || !aligned(dY, of_y)) return DG_ERR_INVALID_ARG;
    if (dR_out == dR || dR_out == R || dR_out == dN || dR_out == Y || dR_out == dY) return DG_ERR_INVALID_ARG;
    if (dY && (dY == Y || dY == R || dY == dR || dY == dN)) return DG_ERR_INVALID_ARG;
    if ((pre || post) && !alone && bad(workspace, 16)) return DG_ERR_INVALID_ARG;
    const bool rb = r_dtype == DG_IN_BF16, yb = dtype == DG_IN_BF16, whole = H % 8 == 0;
    const bool wide = norm_wide(H, most);
    const int threads = norm_threads(H, most);
    dg::NormBwdArgs a{dR, dN, pre ? R : nullptr, Y, w_post, gate, w_pre, dR_out, dY, token ? dgate : nullptr,
                      part_pre, part_post, eps, 1.0 / double(H), alpha, int(T), int(H), gate_kind,
                      threads / 64};
    const auto kernel = rb ? (yb ? norm_bwd_kernel<true, true>(whole, wide) : norm_bwd_kernel<true, false>(whole, wide))
                           : (yb ? norm_bwd_kernel<false, true>(whole, wide) : norm_bwd_kernel<false, false>(whole, wide));
    const int st1 = launch(kernel, a, nb, threads * groups, stream);
    if (st1 != DG_OK) return st1;
  }
  if ((!pre && !post) || alone) return DG_OK;
  // (without rows the sums are zeros)
  const int blocks = int(ceil_div(H, 32));
  dg::NormColumnsArgs c{part_pre, part_post, w_post, channel ? gate : nullptr, dw_pre, dw_post, channel ? dgate : nullptr,
                        int(nb), int(H), pre ? blocks : 0};
  return launch(dg::dg_residual_norm_columns, c, blocks * (pre + post), 1024, stream);
}

int64_t dg_grad_norm_workspace(const int64_t* sizes, const int* dtypes, int count) {
  const int64_t chunks = clip_chunks(sizes, dtypes, count);
  return chunks < 0 ? chunks : clip_few(sizes, count) ? 0 : 8 * chunks;
}

int dg_grad_norm(const void* const* grads, const int64_t* sizes, const int* dtypes, int count, float* norm,
                 void* workspace, hipStream_t stream) {
  const int64_t chunks = clip_chunks(sizes, dtypes, count);
  if (chunks < 0) return int(chunks);
  if (bad(norm, 4) || (chunks > 0 && grads == nullptr)) return DG_ERR_INVALID_ARG;
  const bool few = clip_few(sizes, count);
  if (!few && bad(workspace, 8)) return DG_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (sizes[i] > 0 && bad(grads[i], elem(dtypes[i]))) return DG_ERR_INVALID_ARG;
  dg::ClipBatch b{};
  if (few && chunks > 0) {
    b.norm_out = norm;
    return clip_launches(dg::dg_grad_norm_few, b, grads, sizes, dtypes, count, stream, [](dg::ClipTensor&, int) {}, true);
  }
  b.part = static_cast<double*>(workspace);
  const int st = clip_launches(dg::dg_grad_squares, b, grads, sizes, dtypes, count, stream, [](dg::ClipTensor&, int) {});
  if (st != DG_OK) return st;
  dg::ClipNormArgs a{static_cast<const double*>(workspace), chunks, norm};
  return launch(dg::dg_grad_norm_sum, a, 1, dg::kClipNormThreads, stream);
}

int dg_clip_grads(const void* const* grads, const int64_t* sizes, const int* dtypes, int count, const float* norm,
                  float max_norm, void* const* outs, const int* out_dtypes, hipStream_t stream) {
  const int64_t chunks = clip_chunks(sizes, dtypes, count);
  if (chunks < 0) return int(chunks);
  if (bad(norm, 4) || !isfinite(max_norm) || !(max_norm > 0.f)) return DG_ERR_INVALID_ARG;
  if (chunks == 0) return DG_OK;
  if (grads == nullptr || outs == nullptr || out_dtypes == nullptr) return DG_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (!valid_type(out_dtypes[i])) return DG_ERR_INVALID_ARG;
    if (sizes[i] == 0) continue;
    if (bad(grads[i], elem(dtypes[i])) || bad(outs[i], elem(out_dtypes[i]))) return DG_ERR_INVALID_ARG;
    // in place the types are the same
    if (grads[i] == outs[i] && dtypes[i] != out_dtypes[i]) return DG_ERR_INVALID_ARG;
  }
  const int disjoint = clip_disjoint(grads, sizes, dtypes, count, outs, out_dtypes, norm);
  if (disjoint <= 0) return disjoint == 0 ? DG_ERR_INVALID_ARG : DG_ERR_LAUNCH;
  dg::ClipBatch b{};
  b.norm = norm;
  b.max_norm = max_norm;
  return clip_launches(dg::dg_clip_scale, b, grads, sizes, dtypes, count, stream, [&](dg::ClipTensor& t, int i) {
    t.out = outs[i];
    t.out_bf16 = out_dtypes[i] == DG_IN_BF16;
    t.whole = t.whole && aligned(outs[i], 16);
  });
}

}  // extern "C"
