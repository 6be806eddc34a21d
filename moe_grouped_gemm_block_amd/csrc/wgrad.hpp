// Weight gradient of the grouped product from 8-bit activations, gfx950:
//
//   dW_e[n][k] = sum over expert e's rows r of dY[r][n] X[r][k],
//   X[r][k] = S[r][k / 128] dec(Q[r][k])
//
// Q, S are the E4M3 codes and 1 x 128 scales that the forward product read.
// With power-of-two scales every X value is an exact BF16 value, so the
// products of the BF16 matrix cores are exact and only the FP32 sums round; any
// other scale adds one rounding of S dec(Q) to BF16.
//
// The sum runs over the rows, the slow index of both operands.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "moe.hpp"
#include "swiglu.hpp"

namespace dg {

struct WgradArgs {
  const uint16_t* dY;        // [M][N] BF16
  const uint8_t* X;          // [M][K] codes
  const float* sX;           // [M][Kb]
  const int32_t* offs;       // [G + 1]
  const int32_t* counts;     // [G] or null: whole segments
  void* dW;                  // [G][N][K]
  int G, M, N, K, Kb;
  int n_tiles, k_tiles;
  int accumulate;            // dW += instead of dW =
};

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// Expert e's rows, inside [0, M] whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const WgradArgs& p, int e, int& r0, int& r1) {
  r0 = min(max(p.offs[e], 0), p.M);
  const int end = min(max(p.offs[e + 1], r0), p.M);
  r1 = p.counts ? min(end, r0 + max(min(p.counts[e], p.M), 0)) : end;
}

template <bool OUT_BF16>
__device__ __forceinline__ void wgrad_body(const WgradArgs& p) {
  constexpr int BR = 32, BN = 128, BK = 128;
  __shared__ __attribute__((aligned(16))) uint16_t sy[BR][BN], sx[BR][BK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int q = lane >> 4, r16 = lane & 15;
  const int tiles = p.n_tiles * p.k_tiles;
  const int e = blockIdx.x / tiles, tile = blockIdx.x - e * tiles;
  const int n0 = tile / p.k_tiles * BN, k0 = tile % p.k_tiles * BK;
  int r0, r1;
  expert_rows(p, e, r0, r1);

  const int wn = (wave >> 1) * 64, wk = (wave & 1) * 64;
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int xr = tid >> 3, xc = 16 * (tid & 7);
  for (int r = r0; r < r1; r += BR) {
    const int row = r + xr;
    uint4 y[2] = {uint4{0u, 0u, 0u, 0u}, uint4{0u, 0u, 0u, 0u}}, x = uint4{0u, 0u, 0u, 0u};
    float s = 0.f;
    if (row < r1) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (n0 + xc + 8 * h < p.N) y[h] = *reinterpret_cast<const uint4*>(p.dY + size_t(row) * p.N + n0 + xc + 8 * h);
      if (k0 + xc < p.K) {
        x = *reinterpret_cast<const uint4*>(p.X + size_t(row) * p.K + k0 + xc);
        s = p.sX[size_t(row) * p.Kb + (k0 + xc) / 128];
      }
    }
    float v[16];
    decode4(x.x, s, v);
    decode4(x.y, s, v + 4);
    decode4(x.z, s, v + 8);
    decode4(x.w, s, v + 12);
    __syncthreads();
    *reinterpret_cast<uint4*>(&sy[xr][xc]) = y[0];
    *reinterpret_cast<uint4*>(&sy[xr][xc + 8]) = y[1];
#pragma unroll
    for (int h = 0; h < 16; h += 8)
      *reinterpret_cast<uint4*>(&sx[xr][xc + h]) = uint4{pack_bf16x2(v[h], v[h + 1]), pack_bf16x2(v[h + 2], v[h + 3]),
                                                         pack_bf16x2(v[h + 4], v[h + 5]), pack_bf16x2(v[h + 6], v[h + 7])};
    __syncthreads();
    v8bf fy[4], fx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        fy[i][k] = __builtin_bit_cast(__bf16, sy[8 * q + k][wn + 16 * i + r16]);
        fx[i][k] = __builtin_bit_cast(__bf16, sx[8 * q + k][wk + 16 * i + r16]);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[j], fy[i], acc[i][j], 0, 0, 0);
  }

  // acc[i][j] of lane (q, r16): row n0 + wn + 16 i + r16, columns k0 + wk + 16 j + 4 q .. + 3
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + wn + 16 * i + r16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + wk + 16 * j + 4 * q;
      if (n >= p.N || k >= p.K) continue;
      const size_t at = (size_t(e) * p.N + n) * p.K + k;
      v4f v = acc[i][j];
      if constexpr (OUT_BF16) {
        uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dW) + at);
        if (p.accumulate) {
          const uint2 o = *dst;
          v += v4f{__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xFFFF0000u), __uint_as_float(o.y << 16),
                   __uint_as_float(o.y & 0xFFFF0000u)};
        }
        *dst = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      } else {
        v4f* dst = reinterpret_cast<v4f*>(static_cast<float*>(p.dW) + at);
        if (p.accumulate) v += *dst;
        *dst = v;
      }
    }
  }
}

}  // namespace dg
