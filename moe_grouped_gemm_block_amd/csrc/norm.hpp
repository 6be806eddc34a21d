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
// Both passes are bound by memory, with the vector units busy about as long (8192 rows of
// 4096 in BF16: forward 47.5 us, 5.7 TB/s; backward 76 + 5 us, 5.3 TB/s).  A row's waves
// take eight columns per thread; rows of up to 8192 columns stay in registers, so that
// each is read once and written once, and in BF16 the next row is on its way meanwhile
// (without that 67 and 125 us).  Wider rows are read again for each step, out of the
// caches (1024 rows of 20000: 65 and 190 us).  Workgroups go through many rows, so that
// weights stay in registers and the backward pass has few partial sums of the weights'
// gradients to write.  Statistics are not kept for the backward pass, which reads the rows
// anyway.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "common.hpp"
#include "groups.hpp"
#include "moe.hpp"
#include "swiglu.hpp"

namespace dg {

constexpr int kNormColumns = 8;              // columns of a thread
constexpr int kNormMaxThreads = 1024;
constexpr int kNormGroupThreads = 512;        // of a workgroup that takes several rows at a time
constexpr int kNormWideThreads = 512;         // of wider rows: twice the registers a thread
enum NormGate { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };
enum NormCodes { kCodesNone = 0, kCodesPow2 = 1, kCodesAmax = 2 };

// Eight consecutive values of a row as they lie in memory, zeros past its end.  WHOLE:
// rows of a multiple of eight values, which start 16-byte aligned.  Other rows start at
// any element; the hardware reads and writes vectors at any address, only those that the
// row's end cuts go by elements (8192 rows of 4095 in BF16: forward 63 us,
// 164 by elements; backward 125 and 247).
template <bool BF16>
struct Eight {
  uint32_t w[BF16 ? 4 : 8];
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF16) return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else return __uint_as_float(w[i]);
  }
};
typedef u32x4_nt u32x4_any2 __attribute__((aligned(2)));
typedef u32x4_nt u32x4_any4 __attribute__((aligned(4)));

// v without its first d values (0 to 7), zeros behind the others.
template <bool BF16>
__device__ __forceinline__ void drop_values(Eight<BF16>& v, int d) {
  constexpr int N = BF16 ? 4 : 8;
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v.w[i] = d & 1 ? __builtin_amdgcn_alignbit(i + 1 < N ? v.w[i + 1] : 0u, v.w[i], 16) : v.w[i];
    d >>= 1;
  }
#pragma unroll
  for (int step = 1; step < N; step *= 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) v.w[i] = d & step ? (i + step < N ? v.w[i + step] : 0u) : v.w[i];
  }
}

// NT: as non-temporal loads (what is read once).
template <bool BF16, bool WHOLE, bool NT>
__device__ __forceinline__ Eight<BF16> load_eight(const void* src, size_t row, int c, int H) {
  typedef typename std::conditional<WHOLE, u32x4_nt, typename std::conditional<BF16, u32x4_any2, u32x4_any4>::type>::type V;
  constexpr int N = BF16 ? 4 : 8;
  Eight<BF16> v;
#pragma unroll
  for (int i = 0; i < N; ++i) v.w[i] = 0u;
  if (c >= H) return v;
  // the row's last eight where its end cuts these
  const int from = WHOLE ? c : min(c, H - 8);
  if (WHOLE || from >= 0) {
    const char* at = static_cast<const char*>(src) + (row + from) * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const V* const vec = reinterpret_cast<const V*>(at + 4 * i);
      const u32x4_nt w = NT ? __builtin_nontemporal_load(vec) : *vec;
      v.w[i] = w.x;
      v.w[i + 1] = w.y;
      v.w[i + 2] = w.z;
      v.w[i + 3] = w.w;
    }
    if (!WHOLE && from != c) drop_values(v, c - from);
    return v;
  }
  // a row of less than eight
#pragma unroll 1
  for (int i = H - 1; i >= c; --i) {
    if constexpr (BF16) {
#pragma unroll
      for (int j = N - 1; j > 0; --j) v.w[j] = __builtin_amdgcn_alignbit(v.w[j], v.w[j - 1], 16);
      v.w[0] = v.w[0] << 16 | static_cast<const uint16_t*>(src)[row + i];
    } else {
#pragma unroll
      for (int j = N - 1; j > 0; --j) v.w[j] = v.w[j - 1];
      v.w[0] = static_cast<const uint32_t*>(src)[row + i];
    }
  }
  return v;
}

// Keeps the compiler from holding what it has derived from v in registers until v is used
// again.
template <bool BF16>
__device__ __forceinline__ void derive_again(Eight<BF16>& v) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 4 : 8); ++i) asm volatile("" : "+v"(v.w[i]));
}

__device__ __forceinline__ void derive_again(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(v[i]));
}

// Weights, as values.
template <bool WHOLE>
__device__ __forceinline__ void load8(const float* src, size_t row, int c, int H, float (&v)[8]) {
  const Eight<false> e = load_eight<false, WHOLE, false>(src, row, c, H);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e[i];
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store8(void* dst, size_t row, int c, int H, const float (&v)[8]) {
  typedef typename std::conditional<WHOLE, u32x4_nt, typename std::conditional<BF16, u32x4_any2, u32x4_any4>::type>::type V;
  if (c >= H) return;
  if (WHOLE || c + 8 <= H) {
    char* at = static_cast<char*>(dst) + (row + c) * (BF16 ? 2 : 4);
    if constexpr (BF16) {
      __builtin_nontemporal_store(u32x4_nt{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                           pack_bf16x2(v[6], v[7])}, reinterpret_cast<V*>(at));
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        __builtin_nontemporal_store(u32x4_nt{__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                                             __float_as_uint(v[i + 3])}, reinterpret_cast<V*>(at + 4 * i));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) store_values<BF16, 1>(dst, row + c + i, v + i);
  }
}

// Sums over a row's `waves` waves, in their order; `wave` is this one's number among them.
// All waves of the workgroup take part.  `slots` holds two sets of N values
// per wave, which calls take in turns (`turn`): one barrier a call, since whoever writes a
// set again has passed the barrier of the call between, before which it was read.
constexpr int kNormSums = 4;
constexpr int kNormSlots = 2 * kNormSums * kNormMaxThreads / 64;

template <typename T, int N>
__device__ __forceinline__ void row_sums(T (&v)[N], double* slots, int& turn, int wave, int waves) {
  static_assert(N <= kNormSums, "slots");
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = group_sum<64>(v[i]);
  if (waves == 1) return;
  T* mine = reinterpret_cast<T*>(slots + turn * (kNormSlots / 2)) + (int(threadIdx.x >> 6) - wave) * N;
  turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) mine[wave * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = mine[i];
  for (int w = 1; w < waves; ++w) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += mine[w * N + i];
  }
}

// Sums over a row are taken in FP32: 8 terms a thread one after another, 6 steps of a
// wave, up to 16 waves.  Where FP32's range gets in the way (infinite sums; a mean so
// small that subnormal squares count) the row's are taken again in 64 bits, which hold
// every square.  (All in 64 bits from the start: 8192 rows of 4096 in BF16 forward 54
// instead of 47.5 us, the vector units busy 82 % of the time, backward 91 instead of 76.)
__device__ __forceinline__ bool in_range(float sum, float per, float eps) {
  return sum <= 0x1p100f && __builtin_fmaf(sum, per, eps) >= 0x1p-20f;          // (false for NaN)
}
__device__ __forceinline__ float rstd_of(float sum, float per, float eps) {
  return __builtin_amdgcn_rsqf(__builtin_fmaf(sum, per, eps));
}
// (from the hardware's estimate, good to 2^-23, by two steps of Newton's method: codes are
// bound by instructions, of which a square root and a division are many)
__device__ __forceinline__ double rstd_of(double sum, double per, double eps) {
  const double x = __builtin_fma(sum, per, eps);
  double r = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = __builtin_fma(0.5 * r, __builtin_fma(-x * r, r, 1.0), r);
  return x == __builtin_inf() ? 0.0 : r;
}

template <typename A, typename B>
__device__ __forceinline__ float dot8(const A& a, const B& b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(a[i], b[i], s);
  return s;
}
// (one after another by a variable index, so that registers are left for what is about it)
template <typename A, int... I>
__device__ __forceinline__ double eight_at(const A& a, int i, std::integer_sequence<int, I...>) {
  auto r = a[0];
  ((r = i == I ? a[I] : r), ...);
  return r;
}
template <typename A, typename B>
__device__ __forceinline__ double dot8_f64(const A& a, const B& b) {
  constexpr auto all = std::make_integer_sequence<int, 8>{};
  double s = 0.0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) s = __builtin_fma(eight_at(a, i, all), eight_at(b, i, all), s);
  return s;
}

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
  double eps, per;           // per: 1 / H
  float alpha;
  int T, H, Kb, gate_kind;
};

// Codes of eight values n (f: the same as FP32) of a block that 16 lanes share, and its
// scale.  The codes are those of n / s rounded once: FP32 quotients at both ends of a
// bracket of +-2^-20 around n / s (f is within 2^-24 of n, the reciprocal within 2^-22)
// agree about it but for one value in 2^16, which is then divided in 64 bits.  A block whose
// largest is infinite in FP32 has a NaN scale, by which all its codes are NaN.  (8192 rows of
// 4096 in BF16 to codes: 66 us, 44 by memory; the 64-bit arithmetic of the row and its
// sums bounds it.  With all quotients in 64 bits 5 us more.)
template <bool POW2>
__device__ __forceinline__ uint2 encode8(const double (&n)[8], const float (&f)[8], float& s) {
  float amax = 0.f, r;
  if constexpr (POW2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, __builtin_fabsf(f[i]));
    amax = group_max<16>(amax);
    int e = pow2_exponent(amax);
    if (__builtin_expect(e != pow2_exponent(amax * (1.f + 0x1p-20f)) || e != pow2_exponent(amax * (1.f - 0x1p-20f)), 0)) {
      double a = 0.0;                              // (a loop: nothing of it is done ahead)
#pragma unroll 1
      for (int i = 0; i < 8; ++i) a = fmax(a, __builtin_fabs(eight_at(n, i, std::make_integer_sequence<int, 8>{})));
      a = group_max<16>(a);
      e = max(__builtin_amdgcn_frexp_exp(a) - (__builtin_amdgcn_frexp_mant(a) > 0.875 ? 8 : 9), -126);
    }
    e = amax > 0.f ? e : 0;
    s = amax < __builtin_inff() ? pow2f(e) : __builtin_nanf("");
    r = pow2f(-e);
  } else {
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmax(a, __builtin_fabs(n[i]));
    a = group_max<16>(a);
    double q = a * (1.0 / 448.0);                  // and what it lacks
    q = __builtin_fma(__builtin_fma(-q, 448.0, a), 1.0 / 448.0, q);
    s = !(a > 0.0) ? 1.f : float(a) < __builtin_inff() ? float(q) : __builtin_nanf("");
    r = __builtin_amdgcn_rcpf(s);
  }
  const bool far = !(s >= 0x1p-100f);
  const float r_lo = r * (1.f - 0x1p-20f), r_hi = r * (1.f + 0x1p-20f);
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] = hw_codes4(f[4 * j] * r_lo, f[4 * j + 1] * r_lo, f[4 * j + 2] * r_lo, f[4 * j + 3] * r_lo);
    const uint32_t hi = hw_codes4(f[4 * j] * r_hi, f[4 * j + 1] * r_hi, f[4 * j + 2] * r_hi, f[4 * j + 3] * r_hi);
    if (__builtin_expect(w[j] != hi || far, 0)) {
      uint32_t c = 0;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const double q = eight_at(n, 4 * j + i, std::make_integer_sequence<int, 8>{}) / double(s);
        // (a NaN beside the value that was not decided stays NaN)
        c |= (q != q ? hw_codes4(float(q), 0.f, 0.f, 0.f) & 0xFFu : e4m3_of_f64(q)) << (8 * i);
      }
      w[j] = c;
    }
  }
  return uint2{w[0], w[1]};
}

// RB, YB: the stream and the block's output (and n) are BF16, else FP32.  WIDE: rows
// that do not fit the workgroup's registers.  Elements are computed in FP32, where
// codes are wanted in 64 bits: a code turns on values next to a border, and with 64
// bits it is that of the real number.
template <bool RB, bool YB, int CODES, bool WHOLE, bool WIDE>
__device__ __forceinline__ void norm_body(const NormArgs& p) {
  typedef typename std::conditional<CODES != kCodesNone, double, float>::type F;
  __shared__ double slots[kNormSlots];
  int turn = 0;
  const int step = blockDim.x * 8;
  const int c0 = threadIdx.x * 8;
  const bool block = p.Y != nullptr, post = p.w_post != nullptr, channel = p.gate_kind == kGateChannel;
  // alpha gate w_post, and w_pre
  float onto[8], w_pre[8];
  F onto64[CODES != kCodesNone ? 8 : 1];
  auto weights = [&](int c) {
    float g[8];
    if (post) load8<WHOLE>(p.w_post, 0, c, p.H, onto);
    if (channel) load8<WHOLE>(p.gate, 0, c, p.H, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      F o = p.alpha;
      if (post) o *= onto[i];
      if (channel) o *= g[i];
      if constexpr (CODES != kCodesNone) onto64[i] = o;
      else onto[i] = o;
    }
  };
  if (!WIDE) {
    if (block) weights(c0);
    if (p.w_pre) load8<WHOLE>(p.w_pre, 0, c0, p.H, w_pre);
  }
  Eight<RB> r, r_next;
  Eight<YB> y, y_next;
  auto load = [&](uint32_t t, int c, Eight<RB>& r, Eight<YB>& y) {
    r = load_eight<RB, WHOLE, !WIDE>(p.R, size_t(t) * p.H, c, p.H);
    if (block) y = load_eight<YB, WHOLE, !WIDE>(p.Y, size_t(t) * p.H, c, p.H);
  };
  if (!WIDE) load(blockIdx.x, c0, r_next, y_next);
  // (unsigned: the rows after the last may lie past 2^31)
  for (uint32_t t = blockIdx.x; t < uint32_t(p.T); t += gridDim.x) {
    const size_t row = size_t(t) * p.H;
    const F token = p.gate_kind == kGateToken ? p.gate[t] : 1.f;
    if (!WIDE) {
      // the next row is on its way while this one is computed
      r = r_next;
      y = y_next;
      if (t + gridDim.x < uint32_t(p.T)) load(t + gridDim.x, c0, r_next, y_next);
    }
    // squares over the row: of Y, then of R'
    auto mean_rstd = [&](auto narrow, auto wide) -> F {
      if constexpr (CODES == kCodesNone) {
        float sum[1] = {narrow()};
        row_sums(sum, slots, turn, threadIdx.x >> 6, blockDim.x >> 6);
        if (in_range(sum[0], float(p.per), float(p.eps))) return rstd_of(sum[0], float(p.per), float(p.eps));
      }
      double sum[1] = {wide()};
      row_sums(sum, slots, turn, threadIdx.x >> 6, blockDim.x >> 6);
      return F(rstd_of(sum[0], p.per, p.eps));
    };
    auto squares64 = [&](const auto& v) {
      if constexpr (CODES == kCodesNone) return dot8_f64(v, v);
      double s = 0.0;                              // (the only path here, not the rare one)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fma(double(v[i]), double(v[i]), s);
      return s;
    };
    auto over_row = [&](auto f) {
      decltype(f(c0)) sum = 0;
      for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) sum += f(c);
      return sum;
    };
    auto load_y = [&](int c) {
      if (WIDE) y = load_eight<YB, WHOLE, !WIDE>(p.Y, row, c, p.H);
    };
    F by = token;                                  // y's rstd, with the token's gate
    if (block && post)
      by *= mean_rstd([&] { return over_row([&](int c) { load_y(c); return dot8(y, y); }); },
                      [&] { return over_row([&](int c) { load_y(c); return squares64(y); }); });

    // R' of the columns from c on
    F v[8] = {};
    auto stream = [&](int c) {
      if (WIDE) load(t, c, r, y);
      if (WIDE && block) weights(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = r[i];
        if constexpr (CODES != kCodesNone) {
          if (block) v[i] = __builtin_fma(y[i] * by, onto64[i], v[i]);
        } else {
          if (block) v[i] = __builtin_fmaf(y[i] * by, onto[i], v[i]);
        }
      }
    };
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      stream(c);
      if (!block) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = float(v[i]);
      store8<RB, WHOLE>(p.Rout, row, c, p.H, o);
    }
    if (p.w_pre == nullptr) continue;
    auto again = [&](int c) {
      if (WIDE) stream(c);
    };
    const F pre = mean_rstd([&] { return over_row([&](int c) { again(c); return dot8(v, v); }); },
                            [&] { return over_row([&](int c) { again(c); return squares64(v); }); });
    // (whole groups of 16 lanes run every turn of the codes' blocks)
    for (int c = c0; WIDE ? (c & ~127) < p.H : c == c0; c += step) {
      if (WIDE) {
        stream(c);
        load8<WHOLE>(p.w_pre, 0, c, p.H, w_pre);
      }
      F n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = (v[i] * pre) * w_pre[i];   // (0 past the row's end, or NaN: no maximum)
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = float(n[i]);
      if (p.N) store8<YB, WHOLE>(p.N, row, c, p.H, o);
      if constexpr (CODES != kCodesNone) {
        float s;
        const uint2 q = encode8<CODES == kCodesPow2>(n, o, s);
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
  double eps, per;           // per: 1 / H
  float alpha;
  int T, H, gate_kind, waves;   // waves of a row
};

// Elements in FP32; normalised values x rstd are formed first, so that products on the
// way stay in range.
template <bool RB, bool YB, bool WHOLE, bool WIDE>
__device__ __forceinline__ void norm_bwd_body(const NormBwdArgs& p) {
  __shared__ double slots[kNormSlots];
  __shared__ __attribute__((aligned(16))) float columns[WIDE ? 4 : 8 * (WHOLE || (RB && YB) ? kNormMaxThreads : kNormWideThreads)];
  // the next row is on its way while this one is computed, where there are registers for it
  constexpr bool AHEAD = !WIDE && WHOLE && RB && YB;
  int turn = 0;
  // `groups` rows at a time, of `waves` waves each
  const int waves = p.waves, groups = (blockDim.x >> 6) / waves;
  const int group = (threadIdx.x >> 6) / waves, wave = (threadIdx.x >> 6) % waves;
  const int step = blockDim.x * 8;
  const int c0 = (threadIdx.x - group * waves * 64) * 8;
  // whether any row of those at work takes the rare path: its steps wait for all waves
  auto any_row = [&](bool mine) { return groups > 1 && waves > 1 ? __syncthreads_or(mine) != 0 : mine; };
  const bool block = p.Y != nullptr, pre = p.w_pre != nullptr, post = p.w_post != nullptr;   // (post: only with a block)
  const bool channel = p.gate_kind == kGateChannel;
  // column sums: in registers, or for wide rows in the workgroup's own rows of the
  // partial sums, where only the thread that owns a column reads and writes them
  float sum_pre[8], sum_post[8], w_pre[8], onto[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum_pre[i] = sum_post[i] = 0.f;
  const size_t part = size_t(blockIdx.x) * p.H;
  // w_pre, and alpha gate w_post
  auto weights = [&](int c) {
    float g[8];
    if (pre) load8<WHOLE>(p.w_pre, 0, c, p.H, w_pre);
    if (post) load8<WHOLE>(p.w_post, 0, c, p.H, onto);
    if (channel) load8<WHOLE>(p.gate, 0, c, p.H, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float o = p.alpha;
      if (post) o *= onto[i];
      if (channel) o *= g[i];
      onto[i] = o;
    }
  };
  struct Row {
    Eight<RB> x, dr;
    Eight<YB> y, dn;
  } now, next;
  // (rows past the last read as zeros)
  auto load = [&](uint32_t t, int c, Row& v) {
    const size_t row = size_t(t) * p.H;
    const int H = t < uint32_t(p.T) ? p.H : 0;
    if (pre) {
      v.x = load_eight<RB, WHOLE, !WIDE>(p.R, row, c, H);
      v.dn = load_eight<YB, WHOLE, !WIDE>(p.dN, row, c, H);
    }
    if (block) v.y = load_eight<YB, WHOLE, !WIDE>(p.Y, row, c, H);
    if (p.dR) v.dr = load_eight<RB, WHOLE, !WIDE>(p.dR, row, c, H);
  };
  const uint32_t rows = gridDim.x * groups;
  if (WIDE) {
    for (int c = c0; c < p.H; c += step) {
      if (p.part_pre) store8<false, WHOLE>(p.part_pre, part, c, p.H, sum_pre);
      if (p.part_post) store8<false, WHOLE>(p.part_post, part, c, p.H, sum_post);
    }
  } else {
    weights(c0);
    if (AHEAD) load(blockIdx.x * groups + group, c0, next);
  }
  // (unsigned: the rows after the last may lie past 2^31)
  for (uint32_t t0 = blockIdx.x * groups; t0 < uint32_t(p.T); t0 += rows) {
    const uint32_t t = t0 + group;
    const bool there = t < uint32_t(p.T);
    const size_t row = size_t(t) * p.H;
    const int H = there ? p.H : 0;                   // of what is written
    const float token = p.gate_kind == kGateToken && there ? p.gate[t] : 1.f;
    if (AHEAD) {
      now = next;
      if (t0 + rows < uint32_t(p.T)) load(t + rows, c0, next);
    } else if (!WIDE) {
      load(t, c0, now);
    }
    // R'^2, <w_pre dn, R'>, y^2 over the row
    auto sums_of = [&](auto& sums, auto dot) {
      for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
        if (WIDE) {
          load(t, c, now);
          weights(c);
        }
        if (pre) {
          float d[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = now.dn[i] * w_pre[i];
          sums[0] += dot(now.x, now.x);
          sums[1] += dot(d, now.x);
        }
        if (post) sums[2] += dot(now.y, now.y);
      }
      row_sums(sums, slots, turn, wave, waves);
    };
    float a = 0.f, k = 0.f, b = 1.f;                 // rstd of R', its mean <d, R' rstd> rstd, rstd of y
    if (pre || post) {
      const float per = float(p.per), eps = float(p.eps);
      float sums[3] = {0.f, 0.f, 0.f};
      sums_of(sums, [](const auto& u, const auto& v) { return dot8(u, v); });
      const bool near = (!pre || (in_range(sums[0], per, eps) && __builtin_fabsf(sums[1]) <= 0x1p100f)) &&
                        (!post || in_range(sums[2], per, eps));
      if (!any_row(!near)) {
        if (pre) {
          a = rstd_of(sums[0], per, eps);
          k = a * a * (sums[1] * per);
        }
        if (post) b = rstd_of(sums[2], per, eps);
      } else {
        double wide[3] = {0.0, 0.0, 0.0};
        sums_of(wide, [](const auto& u, const auto& v) { return dot8_f64(u, v); });
        if (pre) {
          const double r = rstd_of(wide[0], p.per, p.eps);
          a = float(r);
          k = float(r * r * (wide[1] * p.per));
        }
        if (post) b = float(rstd_of(wide[2], p.per, p.eps));
      }
    }

    if (!WIDE) {
      derive_again(now.x);
      derive_again(now.dn);
      derive_again(now.y);
    }
    // D of the columns from c on
    float D[8];
    auto total = [&](int c) {
      if (WIDE) {
        load(t, c, now);
        weights(c);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        D[i] = p.dR ? now.dr[i] : 0.f;
        if (pre) D[i] = __builtin_fmaf(now.dn[i] * w_pre[i], a, __builtin_fmaf(now.x[i] * a, -k, D[i]));
      }
    };
    auto onto_y = [&](auto dot) {                    // <alpha w_post gate D, y>, without the token's gate
      decltype(dot(D, now.y)) U[1] = {0};
      for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
        if (WIDE) total(c);
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = D[i] * onto[i];
        U[0] += dot(e, now.y);
      }
      row_sums(U, slots, turn, wave, waves);
      return U[0];
    };
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      total(c);
      store8<RB, WHOLE>(p.dRout, row, c, H, D);
      if (p.part_pre) {
        if (WIDE) load8<WHOLE>(p.part_pre, part, c, p.H, sum_pre);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_pre[i] = __builtin_fmaf(now.dn[i], now.x[i] * a, sum_pre[i]);
        if (WIDE) store8<false, WHOLE>(p.part_pre, part, c, p.H, sum_pre);
      }
    }
    if (!block) continue;
    float kb = 0.f;                                  // the token's gate in it
    if (post || p.gate_kind == kGateToken) {
      const float U = onto_y([](const auto& u, const auto& v) { return dot8(u, v); });
      if (!any_row(!(__builtin_fabsf(U) <= 0x1p100f && b >= 0x1p-50f))) {
        if (p.gate_kind == kGateToken && c0 == 0 && there) p.dgate_token[t] = b * U;
        if (post) kb = b * b * (U * float(p.per)) * token;
      } else {
        const double wide = onto_y([](const auto& u, const auto& v) { return dot8_f64(u, v); });
        if (p.gate_kind == kGateToken && c0 == 0 && there) p.dgate_token[t] = float(b * wide);
        if (post) kb = float(double(b) * b * (wide * p.per) * token);
      }
    }
    if (!WIDE) {
      derive_again(now.y);
      derive_again(D);
    }
    const float tb = token * b;
    for (int c = c0; c < p.H; c = WIDE ? c + step : p.H) {
      if (WIDE) total(c);
      float o[8], yh[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        yh[i] = now.y[i] * b;
        o[i] = __builtin_fmaf(yh[i], -kb, (D[i] * onto[i]) * tb);
      }
      store8<YB, WHOLE>(p.dY, row, c, H, o);
      if (p.part_post) {
        if (WIDE) load8<WHOLE>(p.part_post, part, c, p.H, sum_post);
        const float by = p.alpha * token;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_post[i] = __builtin_fmaf(D[i] * by, yh[i], sum_post[i]);
        if (WIDE) store8<false, WHOLE>(p.part_post, part, c, p.H, sum_post);
      }
    }
  }
  if (!WIDE) {
    // over the groups, in their order
    auto store = [&](float* out, float (&sum)[8]) {
      if (groups > 1) {
        __syncthreads();
        float4* at = reinterpret_cast<float4*>(columns) + 2 * threadIdx.x;
        at[0] = float4{sum[0], sum[1], sum[2], sum[3]};
        at[1] = float4{sum[4], sum[5], sum[6], sum[7]};
        __syncthreads();
        if (group != 0) return;
        for (int g = 1; g < groups; ++g) {
          const float* other = columns + 8 * (threadIdx.x + g * waves * 64);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += other[i];
        }
      }
      store8<false, WHOLE>(out, part, c0, p.H, sum);
    };
    if (p.part_pre) store(p.part_pre, sum_pre);
    if (p.part_post) store(p.part_post, sum_post);
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
    // (eight loads on their way at a time, also where the last are fewer)
    for (int b0 = row; b0 < p.nb; b0 += 8 * 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = b0 + 32 * i < p.nb ? part[size_t(b0 + 32 * i) * p.H + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
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
