// The residual stream past a block and the norms before and after it, gfx950.
//
//   rms(v)   rstd(v) = 1 / sqrt(mean of v^2 + eps)
//   after    z = w_post y rstd(y)                 (without w_post: z = y)
//            R' = R + alpha gate z                (gate by channel, by token, or none)
//   before   n = w_pre R' rstd(R')                of R' as it is before its rounding
//
// n goes out as values, as E4M3 codes with one scale per row and 128 columns (what the
// products read), or as both.  Backward, from the stream R' as it was stored, with
// D = dR' + the gradient of the second norm:
//   d = w_pre dn,  D = dR' + rstd (d - R' rstd^2 <d, R'> / H),  dw_pre = sum dn R' rstd
//   e = alpha gate w_post D,  dy = rstd (e - y rstd^2 <e, y> / H)
//   S = sum alpha D y rstd (by tokens, with a token's gate in it):
//       dw_post = gate S,  dgate = w_post S;  a token's gate: <alpha w_post D, y> rstd
//
// A workgroup takes a row, eight columns per thread; rows of up to 8192 columns stay
// in registers, so that each is read once and written once.  Wider rows are read again
// for each step.  Sums over a row are in 64 bits: squares of BF16's and FP32's largest
// values then stay finite, and the statistics are exact for the outputs' purposes.
// Statistics are not kept for the backward pass, which reads the rows anyway.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "groups.hpp"
#include "moe.hpp"
#include "swiglu.hpp"

namespace dg {

constexpr int kNormColumns = 8;              // columns of a thread
constexpr int kNormMaxThreads = 1024;
constexpr int kNormRegisterWidth = kNormColumns * kNormMaxThreads;
enum NormGate { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };
enum NormCodes { kCodesNone = 0, kCodesPow2 = 1, kCodesAmax = 2 };

// Eight consecutive values of a row, zeros past its end.  WHOLE: rows of a multiple of
// eight values, which start 16-byte aligned.
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void load8(const void* src, size_t row, int c, int H, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (c >= H) return;
  if constexpr (WHOLE) {
    load_values<BF16, BF16 ? 8 : 4>(src, row + c, v);
    if constexpr (!BF16) load_values<BF16, 4>(src, row + c + 4, v + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) load_values<BF16, 1>(src, row + c + i, v + i);
  }
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store8(void* dst, size_t row, int c, int H, const float (&v)[8]) {
  if (c >= H) return;
  if constexpr (WHOLE) {
    store_values<BF16, BF16 ? 8 : 4>(dst, row + c, v);
    if constexpr (!BF16) store_values<BF16, 4>(dst, row + c + 4, v + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) store_values<BF16, 1>(dst, row + c + i, v + i);
  }
}

// Sums over the workgroup, in the order of its waves; `slots` holds N values per wave.
template <int N>
__device__ __forceinline__ void block_sums(double (&v)[N], double* slots) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = group_sum<64>(v[i]);
  if (waves == 1) return;
  __syncthreads();                                   // the last sums have been read
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slots[wave * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = slots[i];
    for (int w = 1; w < waves; ++w) v[i] += slots[w * N + i];
  }
}

// Keeps the compiler from holding what it has derived from v (64-bit copies, products)
// in registers until v is used again.
__device__ __forceinline__ void derive_again(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(v[i]));
}

__device__ __forceinline__ double rstd_of(double sum, int H, double eps) { return 1.0 / sqrt(sum / H + eps); }

struct NormArgs {
  const void* R;             // [T][H]
  const void* Y;             // [T][H], or null: no block before
  const float* w_post;       // [H], or null
  const float* gate;         // [H] or [T], or null
  const float* w_pre;        // [H], or null: no norm of the sum
  void* Rout;                // [T][H], with Y
  void* N;                   // [T][H], or null
  uint8_t* Q;                // [T][H] codes, or null
  float* S;                  // [T][Kb]
  double eps;
  float alpha;
  int T, H, Kb, gate_kind;
};

// The next float towards zero, its last bit set if v is no float: rounding that to
// fewer bits is rounding v itself.
__device__ __forceinline__ float round_odd(double v) {
  const float f = float(v);
  uint32_t b = __float_as_uint(f);
  if (double(f) != v) {
    b -= __builtin_fabs(double(f)) > __builtin_fabs(v);
    b |= 1u;
  }
  return __uint_as_float(b);
}

// Codes of eight values n of a block that 16 lanes share, and its scale.
template <bool POW2>
__device__ __forceinline__ uint2 encode8(const double (&n)[8], float& s) {
  double amax = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmax(amax, __builtin_fabs(n[i]));
  amax = group_max<16>(amax);
  s = 1.f;
  if (amax > 0.0) {
    if constexpr (POW2) {
      const int e = __builtin_amdgcn_frexp_exp(amax) - (__builtin_amdgcn_frexp_mant(amax) > 0.875 ? 8 : 9);
      s = pow2f(min(max(e, -126), 126));
    } else {
      s = float(amax / 448.0);
    }
  }
  const double r = s > 0.f ? 1.0 / double(s) : 0.0;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_fmed3f(round_odd(n[i] * r), -448.f, 448.f);
  return uint2{hw_codes4(v[0], v[1], v[2], v[3]), hw_codes4(v[4], v[5], v[6], v[7])};
}

// RB, YB: the stream and the block's output (and n) are BF16, else FP32.  WIDE: rows
// that do not fit the workgroup's registers.  Elements are computed in FP32, where
// codes are wanted in 64 bits: a code turns on values next to a border, and with 64
// bits it is that of the real number.
template <bool RB, bool YB, int CODES, bool WHOLE, bool WIDE>
__device__ __forceinline__ void norm_body(const NormArgs& p) {
  typedef typename std::conditional<CODES != kCodesNone, double, float>::type F;
  __shared__ double slots[kNormMaxThreads / 64];
  const int step = blockDim.x * 8;
  const int c0 = threadIdx.x * 8;
  const bool block = p.Y != nullptr, post = p.w_post != nullptr, channel = p.gate_kind == kGateChannel;
  // alpha gate w_post, and w_pre
  F onto[8], w_pre[8];
  auto weights = [&](int c) {
    float w[8], g[8];
    if (post) load8<false, WHOLE>(p.w_post, 0, c, p.H, w);
    if (channel) load8<false, WHOLE>(p.gate, 0, c, p.H, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      F o = p.alpha;
      if (post) o *= w[i];
      if (channel) o *= g[i];
      onto[i] = o;
    }
  };
  auto weights_pre = [&](int c) {
    float w[8];
    load8<false, WHOLE>(p.w_pre, 0, c, p.H, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w_pre[i] = w[i];
  };
  if (!WIDE) {
    if (block) weights(c0);
    if (p.w_pre) weights_pre(c0);
  }
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const size_t row = size_t(t) * p.H;
    float y[8], r[8];
    F by = 1;                                      // y's rstd and the token's gate
    if (block) {
      if (!WIDE) load8<YB, WHOLE>(p.Y, row, c0, p.H, y);
      if (!WIDE) load8<RB, WHOLE>(p.R, row, c0, p.H, r);
      if (post) {
        double sum[1] = {0.0};
        for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
          if (WIDE) load8<YB, WHOLE>(p.Y, row, c, p.H, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] += double(y[i]) * y[i];
        }
        block_sums(sum, slots);
        by = F(rstd_of(sum[0], p.H, p.eps));
      }
    } else if (!WIDE) {
      load8<RB, WHOLE>(p.R, row, c0, p.H, r);
    }
    const F token = p.gate_kind == kGateToken ? p.gate[t] : 1.f;

    // R' of the columns from c on
    F v[8] = {};
    auto stream = [&](int c) {
      if (WIDE) load8<RB, WHOLE>(p.R, row, c, p.H, r);
      if (WIDE && block) {
        load8<YB, WHOLE>(p.Y, row, c, p.H, y);
        weights(c);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = r[i];
        if (block) v[i] += (y[i] * by) * (onto[i] * token);
      }
    };
    double sum[1] = {0.0};
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      stream(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += double(v[i]) * double(v[i]);
      if (block) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = float(v[i]);
        store8<RB, WHOLE>(p.Rout, row, c, p.H, o);
      }
    }
    if (p.w_pre == nullptr) continue;
    block_sums(sum, slots);
    const F pre = F(rstd_of(sum[0], p.H, p.eps));
    // (whole groups of 16 lanes run every turn of the codes' blocks)
    for (int c = c0; WIDE ? (c & ~127) < p.H : c == c0; c += step) {
      if (WIDE) {
        stream(c);
        weights_pre(c);
      }
      F n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = c < p.H ? (v[i] * pre) * w_pre[i] : F(0);
      if (p.N) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = float(n[i]);
        store8<YB, WHOLE>(p.N, row, c, p.H, o);
      }
      if constexpr (CODES != kCodesNone) {
        float s;
        const uint2 q = encode8<CODES == kCodesPow2>(n, s);
        if (c < p.H) {
          *reinterpret_cast<uint2*>(p.Q + row + c) = q;
          if ((threadIdx.x & 15) == 0) p.S[size_t(t) * p.Kb + c / 128] = s;
        }
      }
    }
  }
}

// ---- backward -----------------------------------------------------------------------
struct NormBwdArgs {
  const void* dR;            // [T][H], or null: zeros
  const void* dN;            // [T][H], with w_pre
  const void* R;             // [T][H] the stream after the block; null without w_pre
  const void* Y;             // [T][H], or null
  const float* w_post;
  const float* gate;
  const float* w_pre;
  void* dRout;               // [T][H]
  void* dY;                  // [T][H], with Y
  float* dgate_token;        // [T], with a token's gate
  float* part_pre;           // [gridDim.x][H], with w_pre
  float* part_post;          // [gridDim.x][H], with w_post or a channel's gate
  double eps;
  float alpha;
  int T, H, gate_kind;
};

// Elements in FP32; normalised values x rstd are formed first, so that products on the
// way stay in range.
template <bool RB, bool YB, bool WHOLE, bool WIDE>
__device__ __forceinline__ void norm_bwd_body(const NormBwdArgs& p) {
  __shared__ double slots[3 * kNormMaxThreads / 64];
  const int step = blockDim.x * 8;
  const int c0 = threadIdx.x * 8;
  const bool block = p.Y != nullptr, pre = p.w_pre != nullptr, post = p.w_post != nullptr;
  const bool channel = p.gate_kind == kGateChannel;
  // column sums: in registers, or for wide rows in the workgroup's own rows of the
  // partial sums, where only the thread that owns a column reads and writes them
  float sum_pre[8], sum_post[8], w_pre[8], onto[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum_pre[i] = sum_post[i] = 0.f;
  const size_t part = size_t(blockIdx.x) * p.H;
  // w_pre, and alpha gate w_post
  auto weights = [&](int c) {
    float w[8], g[8];
    if (pre) load8<false, WHOLE>(p.w_pre, 0, c, p.H, w_pre);
    if (post) load8<false, WHOLE>(p.w_post, 0, c, p.H, w);
    if (channel) load8<false, WHOLE>(p.gate, 0, c, p.H, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float o = p.alpha;
      if (post) o *= w[i];
      if (channel) o *= g[i];
      onto[i] = o;
    }
  };
  if (WIDE) {
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      if (p.part_pre) store8<false, false>(p.part_pre, part, c, p.H, sum_pre);
      if (p.part_post) store8<false, false>(p.part_post, part, c, p.H, sum_post);
    }
  } else {
    weights(c0);
  }
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const size_t row = size_t(t) * p.H;
    float x[8] = {}, y[8] = {}, dn[8] = {}, D[8];
    auto load = [&](int c) {
      if (WIDE) weights(c);
      if (pre) {
        load8<RB, WHOLE>(p.R, row, c, p.H, x);
        load8<YB, WHOLE>(p.dN, row, c, p.H, dn);
      }
      if (block) load8<YB, WHOLE>(p.Y, row, c, p.H, y);
      if (p.dR) {
        load8<RB, WHOLE>(p.dR, row, c, p.H, D);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) D[i] = 0.f;
      }
    };
    if (!WIDE) load(c0);
    double sums[3] = {0.0, 0.0, 0.0};                // R'^2, <w_pre dn, R'>, y^2
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      if (WIDE) load(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (pre) {
          sums[0] += double(x[i]) * x[i];
          sums[1] += double(dn[i] * w_pre[i]) * x[i];
        }
        if (block && post) sums[2] += double(y[i]) * y[i];
      }
    }
    if (!WIDE) {
      derive_again(x);
      derive_again(y);
      derive_again(dn);
    }
    if (pre || (block && post)) block_sums(sums, slots);
    double a = 0.0, k = 0.0, b = 1.0;
    if (pre) {
      a = rstd_of(sums[0], p.H, p.eps);
      k = a * a * sums[1] / p.H;
    }
    if (block && post) b = rstd_of(sums[2], p.H, p.eps);
    const float a_ = float(a), k_ = float(k), b_ = float(b);
    const float token = p.gate_kind == kGateToken ? p.gate[t] : 1.f;

    auto total = [&](int c) {
      if (WIDE) load(c);
      if (!pre) return;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= a_;
        D[i] += (dn[i] * w_pre[i]) * a_ - x[i] * k_;
      }
    };
    double U[1] = {0.0};                             // <alpha w_post gate D, y>, without the token's gate
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      total(c);
      store8<RB, WHOLE>(p.dRout, row, c, p.H, D);
      if (block) {
#pragma unroll
        for (int i = 0; i < 8; ++i) U[0] += double(D[i] * onto[i]) * y[i];
      }
      if (p.part_pre) {
        if (WIDE) load8<false, false>(p.part_pre, part, c, p.H, sum_pre);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_pre[i] = __builtin_fmaf(dn[i], x[i], sum_pre[i]);
        if (WIDE) store8<false, false>(p.part_pre, part, c, p.H, sum_pre);
      }
    }
    if (!block) continue;
    if (post || p.gate_kind == kGateToken) block_sums(U, slots);
    if (p.gate_kind == kGateToken && threadIdx.x == 0) p.dgate_token[t] = float(b * U[0]);
    const float kb = post ? float(b * b * U[0] / p.H) : 0.f;
    const float scale = p.alpha * token;
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      if (WIDE) total(c);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yh = y[i] * b_;
        o[i] = token * ((D[i] * onto[i]) * b_ - yh * kb);
        y[i] = yh;
      }
      store8<YB, WHOLE>(p.dY, row, c, p.H, o);
      if (p.part_post) {
        if (WIDE) load8<false, false>(p.part_post, part, c, p.H, sum_post);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_post[i] = __builtin_fmaf(scale * D[i], y[i], sum_post[i]);
        if (WIDE) store8<false, false>(p.part_post, part, c, p.H, sum_post);
      }
    }
  }
  if (!WIDE) {
    if (p.part_pre) store8<false, WHOLE>(p.part_pre, part, c0, p.H, sum_pre);
    if (p.part_post) store8<false, WHOLE>(p.part_post, part, c0, p.H, sum_post);
  }
}

// Column sums over the workgroups' partial rows, in their order: 32 columns a
// workgroup of 1024 threads, 32 threads a column.
struct NormColumnsArgs {
  const float* part_pre;     // [nb][H], or null
  const float* part_post;    // [nb][H], or null
  const float* w_post;       // [H], or null
  const float* gate;         // [H] by channel, or null
  float* dw_pre;             // [H]
  float* dw_post;            // [H], or null
  float* dgate;              // [H], or null
  int nb, H, blocks;         // workgroups of part_pre; the others take part_post
};

__device__ __forceinline__ void norm_columns_body(const NormColumnsArgs& p) {
  __shared__ float sums[32][33];
  const bool second = int(blockIdx.x) >= p.blocks;
  const int block = second ? blockIdx.x - p.blocks : blockIdx.x;
  const float* part = second ? p.part_post : p.part_pre;
  const int col = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = block * 32 + col;
  float s = 0.f;
  if (c < p.H) {
    for (int b = row; b < p.nb; b += 32) s += part[size_t(b) * p.H + c];
  }
  sums[row][col] = s;
  __syncthreads();
  if (row != 0 || c >= p.H) return;
  for (int i = 1; i < 32; ++i) s += sums[i][col];
  if (!second) {
    p.dw_pre[c] = s;
    return;
  }
  if (p.dw_post) p.dw_post[c] = p.gate ? s * p.gate[c] : s;
  if (p.dgate) p.dgate[c] = p.w_post ? s * p.w_post[c] : s;
}

}  // namespace dg
