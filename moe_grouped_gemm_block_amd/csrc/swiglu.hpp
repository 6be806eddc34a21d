// The gated activation between an expert's two products, with its input kept
// in 8 bits for the backward pass, gfx950.
//
//   h = [g | u] (one row of the first product), a = u g / (1 + e^-g)
//   forward   A, sA = codes and scales of a      (the second product's operand)
//             Hq, sH = codes and scales of g and of u   (the checkpoint)
//   backward  from g, u as the checkpoint holds them, p = 1 / (1 + e^-g):
//             dg = dA u p (1 + g (1 - p)),  du = dA g p
//
// Scales are powers of two, one per row and 128 columns of a, g and u each:
// moving a float by a power of two does not round, so the only rounding of the
// checkpoint is the one to E4M3's four significant bits, and decoded values are
// exact BF16 values (which the weight gradient's matrix product relies on).
//
// Both passes are bound by memory: forward 4 bytes in and 3 out per element
// pair (9216 rows of 2 x 4096 in BF16: 45.9 us, 5.8 TB/s; a copy reaches 5.3),
// backward 4 in and 4 out (6.7 TB/s).  An 8-lane group takes one block of 128
// columns, 16 values of g, u and a per lane in registers; the block maxima are
// reduced by lane permutations, nothing goes through LDS.  (Eight values per
// lane and 16 lanes, for more waves in flight: 48.8 us.)
//
// The codes of a are those of the real number u g / (1 + e^-g) rounded once, not
// of its FP32 approximation: a fast FP32 value within 2^-21 of it is encoded at
// both ends of a bracket of +-2^-20, and where the two codes differ (about one
// value in 2^16) or FP32's range gets in the way, it is computed again in
// double.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "moe.hpp"
#include "quant.hpp"

namespace dg {

struct SwigluArgs {
  const void* H;         // [M][2 I]
  uint8_t* A;            // [M][I] codes
  float* sA;             // [M][Ib]
  uint8_t* Hq;           // [M][2 I] codes, or null: no checkpoint
  float* sH;             // [M][2][Ib]
  int M, I, Ib;
};

// e^-g within 2^-22 of it: the exponent's product with log2(e) keeps its
// rounding error as a second term (FP32's alone would cost |g| 2^-24).  Gates
// count as at least -80, where e^-g comes near FP32's end, and at most 150, where
// it is 0 and the largest gates' exponents would overflow.
__device__ __forceinline__ float exp_neg(float g) {
  g = __builtin_amdgcn_fmed3f(g, -80.f, 150.f);
  constexpr float L = 1.44269504088896341f, L_LO = 1.92596299e-8f;   // log2(e) = L + L_LO
  const float hi = -g * L;
  const float lo = __builtin_fmaf(-g, L, -hi) - g * L_LO;
  const float e = __builtin_amdgcn_exp2f(hi);
  return __builtin_fmaf(e, lo * 0.693147180559945f, e);
}

__device__ __forceinline__ double silu_mul_f64(float g, float u) {
  const double gd = g;
  return double(u) * (gd / (1.0 + exp(-gd)));
}

// u g / (1 + e^-g) within 2^-21 for g >= -80 (results outside FP32's normal range
// aside)
__device__ __forceinline__ float silu_mul(float g, float u) {
  return u * (g * __builtin_amdgcn_rcpf(1.f + exp_neg(g)));
}

// E4M3 code of v (|v| <= 448 or a little above it), rounded once.
__device__ __forceinline__ uint32_t e4m3_of_f64(double v) {
  const double m = fmin(__builtin_fabs(v), 448.0);
  const int e = max(__builtin_amdgcn_frexp_exp(m), -5);       // v = [0.5, 1) 2^e; grid step 2^(e - 4)
  const float q = float(__builtin_ldexp(__builtin_rint(__builtin_ldexp(m, 4 - e)), e - 4));
  return hw_codes4(float(__builtin_copysign(double(q), v)), 0.f, 0.f, 0.f) & 0xFFu;
}

template <bool IN_BF16, bool CHECKPOINT>
__device__ __forceinline__ void swiglu_body(const SwigluArgs& p) {
  const int lane = threadIdx.x & 63;
  uint32_t m;
  int ib;
  row_and_place<32>(threadIdx.x >> 3, p.Ib, m, ib);
  const int col = ib * 128 + 16 * (lane & 7);
  const bool in = m < uint32_t(p.M) && col < p.I;
  Q1Buf<IN_BF16> bg, bu;
  const size_t e0 = in ? size_t(m) * 2 * p.I + col : 0;
  load_q16(bg, p.H, e0, in);
  load_q16(bu, p.H, e0 + (in ? p.I : 0), in);
  float a[16], ga = 0.f, ua = 0.f, aa = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float g = q1_value(bg, i), u = q1_value(bu, i);
    a[i] = silu_mul(g, u);
    ga = fmaxf(ga, __builtin_fabsf(g));
    ua = fmaxf(ua, __builtin_fabsf(u));
  }
  if (__builtin_expect(ga > 80.f, 0)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float g = q1_value(bg, i);
      if (g < -80.f) a[i] = float(silu_mul_f64(g, q1_value(bu, i)));
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) aa = fmaxf(aa, __builtin_fabsf(a[i]));
  aa = group8_max(aa);
  ga = group8_max(ga);
  ua = group8_max(ua);
  if constexpr (CHECKPOINT) {
    float sg, su;
    const Codes16 cg = encode16<true>([&](int i) { return q1_value(bg, i); }, ga, sg);
    const Codes16 cu = encode16<true>([&](int i) { return q1_value(bu, i); }, ua, su);
    if (in) {
      store16<false>(p.Hq + e0, u32x4_nt{cg.w[0], cg.w[1], cg.w[2], cg.w[3]});
      store16<false>(p.Hq + e0 + p.I, u32x4_nt{cu.w[0], cu.w[1], cu.w[2], cu.w[3]});
    }
    if (m < uint32_t(p.M) && (lane & 7) == 0) {
      p.sH[(size_t(m) * 2) * p.Ib + ib] = sg;
      p.sH[(size_t(m) * 2 + 1) * p.Ib + ib] = su;
    }
  }

  // the scale of a's block, from the maximum in reals (which FP32 may have lost)
  int e = 0;
  bool some = ga > 0.f && ua > 0.f, all64 = false;
  if (some) {
    e = pow2_exponent(aa * (1.f - 0x1p-20f));
    all64 = aa < 0x1p-81f;                // values near FP32's lower end: no bracket is trusted
    if (all64 || e != pow2_exponent(aa * (1.f + 0x1p-20f))) {
      double md = 0.0;
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {    // registers are not indexed by a variable
          g = i == k ? q1_value(bg, k) : g;
          u = i == k ? q1_value(bu, k) : u;
        }
        md = fmax(md, __builtin_fabs(silu_mul_f64(g, u)));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) md = fmax(md, __shfl_xor(md, o, 64));
      const double mant = __builtin_amdgcn_frexp_mant(md);
      e = max(__builtin_amdgcn_frexp_exp(md) - (mant > 0.875 ? 8 : 9), -126);
      some = md > 0.0;
    }
  }
  const float s = some ? pow2f(e) : 1.f, r = some ? pow2f(-e) : 1.f;
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float r_lo = r * (1.f - 0x1p-20f), r_hi = r * (1.f + 0x1p-20f);
    w[j] = hw_codes4(a[4 * j] * r_lo, a[4 * j + 1] * r_lo, a[4 * j + 2] * r_lo, a[4 * j + 3] * r_lo);
    const uint32_t hi = hw_codes4(a[4 * j] * r_hi, a[4 * j + 1] * r_hi, a[4 * j + 2] * r_hi, a[4 * j + 3] * r_hi);
    if (w[j] != hi || all64) {
      uint32_t c = 0;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          g = i == k ? q1_value(bg, 4 * j + k) : g;
          u = i == k ? q1_value(bu, 4 * j + k) : u;
        }
        c |= e4m3_of_f64(silu_mul_f64(g, u) * double(r)) << (8 * i);
      }
      w[j] = c;
    }
  }
  if (in) store16<false>(p.A + size_t(m) * p.I + col, u32x4_nt{w[0], w[1], w[2], w[3]});
  if (m < uint32_t(p.M) && (lane & 7) == 0) p.sA[size_t(m) * p.Ib + ib] = s;
}

struct SwigluBwdArgs {
  const void* dA;        // [M][I]
  const uint8_t* Hq;     // [M][2 I] codes
  const float* sH;       // [M][2][Ib]
  void* dH;              // [M][2 I]
  int M, I, Ib;
};

typedef float v2f __attribute__((ext_vector_type(2)));

// Four E4M3 codes -> their values times s.
__device__ __forceinline__ void decode4(uint32_t w, float s, float* v) {
  const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
  v[0] = lo.x * s;
  v[1] = lo.y * s;
  v[2] = hi.x * s;
  v[3] = hi.y * s;
}

// Value of the i-th of eight E4M3 codes.
__device__ __forceinline__ float code_value(uint2 w, int i) {
  return __builtin_amdgcn_cvt_f32_fp8(int((i < 4 ? w.x : w.y) >> (8 * (i & 3))), 0);
}

// The gradient of one pair in double, at any gate: e^-g ends at infinity where p
// ends at 0.
__device__ __forceinline__ void silu_mul_bwd_f64(float d, double g, double u, float& dg_, float& du) {
  const double pr = 1.0 / (1.0 + exp(-g)), x = g * pr;
  du = float(d * x);
  dg_ = float(d * (u * (x * (1.0 - pr) + pr)));
}

// A thread takes 8 columns: 8 codes of g and of u and 8 values of dA in, 8
// values of dg and of du out.  FP32, one rounding to the output type; gates below
// -56, whose factors go to 0 with e^g, in double (only blocks with a scale above
// 1/8 reach them, 448 / 8 = 56, so others are not searched).  NaN goes through
// either: comparisons that choose are false for it, and nothing clamps.
// dA and dH past the caches (non-temporal), the codes' pieces of 8 bytes not: 9216
// rows of 2 x 4096 in BF16 45.4 us, 6.7 TB/s (all plain 52.7, all non-temporal
// 47.4).
template <bool BF16>
__device__ __forceinline__ void swiglu_bwd_body(const SwigluBwdArgs& p) {
  uint32_t m;
  int col;
  row_and_place<256>(threadIdx.x, p.I / 8, m, col);
  if (m >= uint32_t(p.M)) return;
  col *= 8;
  const size_t h0 = size_t(m) * 2 * p.I + col;
  const uint2 wg = *reinterpret_cast<const uint2*>(p.Hq + h0);
  const uint2 wu = *reinterpret_cast<const uint2*>(p.Hq + h0 + p.I);
  const float sg = p.sH[(size_t(m) * 2) * p.Ib + col / 128], su = p.sH[(size_t(m) * 2 + 1) * p.Ib + col / 128];
  float g[8], u[8], d[8], dg_[8], du[8];
  decode4(wg.x, sg, g);
  decode4(wg.y, sg, g + 4);
  decode4(wu.x, su, u);
  decode4(wu.y, su, u + 4);
  constexpr int V = BF16 ? 8 : 4;
#pragma unroll
  for (int v = 0; v < 8; v += V) load_values<BF16, V, true>(p.dA, size_t(m) * p.I + col + v, d + v);
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    // p = 1 / (1 + e) and 1 - p = e p, which keeps its relative precision where
    // p is near 1
    const float e = exp_neg(g[v]);
    const float pr = __builtin_amdgcn_rcpf(1.f + e);
    const float x = g[v] * pr;
    du[v] = d[v] * x;
    dg_[v] = d[v] * (u[v] * __builtin_fmaf(x, e * pr, pr));
  }
  // Blocks with smaller or larger scales are in double as a whole: with these, g p
  // and u (p + g p (1 - p)) are normal numbers before dA comes to them (gates of
  // at least -56: p >= 2^-81 and u >= 2^-49; where p is near 1/2, g >= 2^-109), so
  // that only the results themselves can leave FP32's range.  Gates whose codes
  // round up past its end are infinite here, and far.
  const bool g_out = !(sg >= 0x1p-100f), u_out = !(su >= 0x1p-40f && su <= 0x1p100f);
  bool far = g_out || u_out;
  if (__builtin_expect(!(sg <= 0.125f), 0)) {
#pragma unroll
    for (int v = 0; v < 8; ++v) far |= !(g[v] >= -56.f && g[v] <= __FLT_MAX__);
  }
#pragma unroll
  for (int v = 0; v < 8; v += V) {
    store_values<BF16, V>(p.dH, h0 + v, dg_ + v);
    store_values<BF16, V>(p.dH, h0 + p.I + v, du + v);
  }
  // over what is stored already, which keeps the values above out of registers
  if (__builtin_expect(far, 0)) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const double gd = double(code_value(wg, i)) * double(sg);
      const bool ordinary = gd >= -56.0 && gd <= __FLT_MAX__ && !g_out;
      if (ordinary && !u_out) continue;
      float di, a, b;
      load_values<BF16, 1>(p.dA, size_t(m) * p.I + col + i, &di);
      silu_mul_bwd_f64(di, gd, double(code_value(wu, i)) * double(su), a, b);
      store_values<BF16, 1>(p.dH, h0 + i, &a);
      if (!ordinary) store_values<BF16, 1>(p.dH, h0 + p.I + i, &b);
    }
  }
}

}  // namespace dg
