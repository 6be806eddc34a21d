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
// The sum runs over the rows, the slow index of both operands, so every operand
// of the matrix cores is a transposed read (ds_read_b64_tr_b16).  A workgroup of
// four waves takes a 256 x 128 tile of dW_e (128 x 128 where those would leave
// CUs idle) and all rows of the expert, 32 per step; two workgroups share a CU,
// so that one's products cover the other's waits and stores.  dY goes straight
// into LDS; X goes there as codes, each thread's own 16 bytes and scale, two
// steps later through registers and back as BF16, one conversion per element and
// tile.  Copies are issued three steps (dY) and five (X) ahead into rotating slots;
// each lands by the end of the step after the one that issued it.
//
// The results leave through LDS in whole lines and past the caches (non-temporal
// stores), which keeps the operands in L2: 8 experts of 1024 rows with FP32
// results 333 -> 318 us, 64 uneven experts with BF16 results 277 -> 258 us
// (non-temporal stores of half lines were slower, 353 and 295).
//
// What bounds it.  8 experts of 1024 rows, N = K = 4096: 311 to 322 us with FP32
// results (850 to 885 TFLOP/s), 282 to 289 with BF16 ones.  That is nearly the sum
// of the stores (94 and 46 us without rows) and of the products (further rows cost
// 1.23 PFLOP/s): a tile's stores overlap little with other tiles' products.  The
// matrix units are busy 0.4 of the cycles.  Zeros as operands save 40 us, by the
// clock, which falls from 2.1 to 1.85 GHz over nine launches; a workgroup made to
// wait between its stores, or to start later, changes nothing.  A library's products
// of BF16 operands of this shape take 303 to 315 us one after another with BF16
// results, 358 to 369 with FP32 ones, 263 to 271 batched on operands laid out for
// it.  64 experts with 16384 rows unevenly, N = K = 2048, BF16: 243 to 270 us by
// their routing, most tiles having two to eight steps: the first loads and the
// stores of a tile, covered by one other workgroup only.  Few tiles: 64 of 128 x 128
// with 1024 rows 16.7 us, with 16384 rows 194, the same as 16 or 128 tiles, since a
// workgroup takes all rows.  Added to FP32 gradients instead of stored: 452 us.
//
// What was slower: 128 x 128 tiles, plain LDS reads and one stage 967 and 627 us
// (8 and 64 experts); one workgroup of 256 x 256 tiles per CU, with a third less LDS
// traffic, 340 and 303; 512 workgroups that go through shares of the tiles, loading
// the next one before the stores of the last, 329 and 304 (where rows are even, 134
// instead of 151 us for 256 each); the experts in order of their rows, the same on
// average.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "gemm_sharedb.hpp"
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
  int per_xcd;               // tiles of an expert per XCD, or 0: experts' tiles in a row
  int accumulate;            // dW += instead of dW =
};

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// Expert e's rows, inside [0, M] whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const WgradArgs& p, int e, int& r0, int& r1) {
  // three loads at once: without counts the third reads the offset again
  const int32_t* c = p.counts ? p.counts : p.offs;
  const int o0 = p.offs[e], o1 = p.offs[e + 1], n = c[e];
  r0 = min(max(o0, 0), p.M);
  const int end = min(max(o1, r0), p.M);
  r1 = p.counts ? min(end, r0 + max(min(n, p.M - r0), 0)) : end;
}

// The tile of a workgroup; false: none.  Workgroup b runs on XCD b % 8.  With
// many tiles per expert each XCD takes a contiguous eighth of every expert's
// tiles, so that its L2 serves their common operands and uneven experts load all
// XCDs alike; the last eighth may be short.
__device__ __forceinline__ bool tile_of_expert(const WgradArgs& p, int& e, int& tile) {
  const int tiles = p.n_tiles * p.k_tiles, b = blockIdx.x;
  if (p.per_xcd == 0) {
    e = b / tiles;
    tile = b - e * tiles;
    return true;
  }
  const int i = b >> 3;
  e = i / p.per_xcd;
  tile = (b & 7) * p.per_xcd + (i - e * p.per_xcd);
  return tile < tiles;
}

// Tiles run along pairs of tiles of N: what an XCD has in flight shares few
// columns of dY, whose tiles are four times X's in bytes.
__device__ __forceinline__ void tile_at(const WgradArgs& p, int tile, int& tn, int& tk) {
  const int pair = tile / (2 * p.k_tiles), rest = tile - pair * 2 * p.k_tiles;
  const bool two = 2 * pair + 1 < p.n_tiles;
  tk = two ? rest >> 1 : rest;
  tn = 2 * pair + (two ? rest & 1 : 0);
}

// Four values of each of 16 columns from LDS, transposed on the way: the
// 16 lanes of a group read a 4 x 16 block (lane i: row i / 4, columns
// 4 (i % 4) .. + 3, 8 bytes) and lane i gets column i of its four rows
// (ds_read_b64_tr_b16).
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
__device__ __forceinline__ v4s read_tr(lds_u8* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
}

// Four E4M3 codes times s -> four BF16.  With a power of two the FP32 product is
// a BF16 value already; with any other scale it rounds once more.
__device__ __forceinline__ uint2 decode4_bf16(uint32_t c, float s) {
  float v[4];
  decode4(c, s, v);
  return uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

template <int BN, int BK, bool OUT_BF16>
__device__ __forceinline__ void wgrad_body(const WgradArgs& p) {
  constexpr int BR = 32;                         // rows per step: one MFMA deep
  constexpr int NI = BN / 32, KI = BK / 32;      // 16 x 16 MFMA tiles per wave
  constexpr int YROW = 2 * BN, XROW = 2 * BK;    // bytes of an LDS row
  constexpr int YB = BR * YROW, XB = BR * XROW;  // bytes of a stage
  constexpr int YC = YB / 4096;                  // copies of 1 KB per wave and stage
  constexpr int RB = 4096, SB = 1024;            // codes and scales of a stage
  static_assert(BR * BK == RB, "a thread takes 16 codes and their scale");
  static_assert(KI == 4, "the step's schedule");
  constexpr int DEPTH = kSingleStage ? 1 : 3;    // stages of everything copied
  constexpr int X0 = DEPTH * YB, R0 = X0 + (kSingleStage ? 1 : 2) * XB, S0 = R0 + DEPTH * RB;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S0 + DEPTH * SB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, r16 = lane & 15;

  int e, tile;
  if (!tile_of_expert(p, e, tile)) return;
  int tn, tk;
  tile_at(p, tile, tn, tk);
  const int n0 = tn * BN, k0 = tk * BK;
  int r0, r1;
  expert_rows(p, e, r0, r1);
  r0 = __builtin_amdgcn_readfirstlane(r0);
  r1 = __builtin_amdgcn_readfirstlane(r1);
  const int full = (r1 - r0) / BR, last = (r1 - r0) % BR, steps = full + (last > 0);
  const int N = p.N, K = p.K, Kb = p.Kb;
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>((lds_u8*)lds));

  // Buffer size of a step's rows, from the tile's first column to the end of the
  // last row: rows past the expert's read zeros.  All but the last steps have BR
  // rows.  (In scalar registers; as a function of s alone it would go through the
  // vector units.)
  struct Sizes {
    uint32_t full, last;
  };
  auto sizes = [&](int width, int first, int elem) {
    return Sizes{uint32_t((BR * width - first) * elem), uint32_t(max(last * width - first, 0) * elem)};
  };
  const Sizes y_size = sizes(N, n0, 2), x_size = sizes(K, k0, 1), s_size = sizes(Kb, k0 / 128, 4);
  auto step_size = [&](const Sizes& z, int s) { return s < full ? z.full : s == full ? z.last : 0u; };

  // ---- dY: copies of 1 KB (512 / BN rows) straight into LDS -----------------
  // Block b (16 columns, 32 bytes) of row r sits at b ^ (r % 8): the transposed
  // reads take one block of 16 consecutive rows, 8 rows per half-wave, which
  // then lie in distinct banks.
  constexpr int YR = 512 / BN;
  const int yr = wave * YR + lane / (64 / YR), yc = lane % (64 / YR);
  const uint32_t y_lane = uint32_t(yr * N + 16 * ((yc >> 1) ^ (yr & 7)) + 8 * (yc & 1)) * 2u;
  auto copy_y = [&](int s, uint32_t slot) {
    const i32x4 rs = make_rsrc(p.dY + (size_t(r0) + size_t(s) * BR) * N + n0, step_size(y_size, s));
#pragma unroll
    for (int c = 0; c < YC; ++c)
      copy16_to_lds(rs, y_lane + uint32_t(c * 4 * YR * N) * 2u, lds0 + slot * YB + uint32_t(c * 4096 + wave * 1024));
  };

  // ---- X: codes and scales copied into LDS, each thread its own, and from there
  // decoded into the matrix cores' operand --------------------------------------
  constexpr int XT = BK / 16;                    // threads per row
  const int xr = tid / XT, xb = tid % XT;
  const uint32_t x_lane = uint32_t(xr * K + 16 * xb);
  const uint32_t s_lane = uint32_t(xr * Kb + xb / 8) * 4u;
  auto copy_x = [&](int s, uint32_t slot) {
    const i32x4 rx = make_rsrc(p.X + (size_t(r0) + size_t(s) * BR) * K + k0, step_size(x_size, s));
    const i32x4 rs = make_rsrc(p.sX + (size_t(r0) + size_t(s) * BR) * Kb + k0 / 128, step_size(s_size, s));
    copy16_to_lds(rx, x_lane, lds0 + R0 + slot * RB + uint32_t(wave * 1024));
    copy4_to_lds(rs, s_lane, lds0 + S0 + slot * SB + uint32_t(wave * 256));
  };
  // Row r of the operand is two planes of 16-byte granules: columns 0 .. 7 of
  // every block of 16 in the first, 8 .. 15 in the second.  Granule b sits at
  // b ^ (r % 8), in the second plane at b ^ (r % 8) ^ 1: eight lanes that
  // store side by side, and the 8 rows x 32 bytes of a transposed read, hit
  // distinct banks.
  uint32_t x_wr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    x_wr[h] = uint32_t(X0 + xr * XROW + h * (XROW / 2) + 16 * (xb ^ (xr & 7) ^ h));
  }
  u32x4 xraw, xdec[2];
  float xs;
  auto read_raw = [&](uint32_t slot) {
    xraw = *reinterpret_cast<const u32x4*>(lds + R0 + slot * RB + 16 * tid);
    xs = *reinterpret_cast<const float*>(lds + S0 + slot * SB + 4 * tid);
  };
  auto decode_word = [&](int w) {
    const uint2 d = decode4_bf16(xraw[w], xs);
    xdec[w >> 1][2 * (w & 1)] = d.x;
    xdec[w >> 1][2 * (w & 1) + 1] = d.y;
  };
  auto write_x = [&](uint32_t stage) {
    uint8_t* st = lds + stage * XB;
    *reinterpret_cast<u32x4*>(st + x_wr[0]) = xdec[0];
    *reinterpret_cast<u32x4*>(st + x_wr[1]) = xdec[1];
  };

  // ---- operand reads: columns 16 f .. + 15 of the wave's part, 32 rows ---------
  // Element 4 h + c of lane (q, r16) is row 16 h + 4 q + c, for both operands.
  const int fr = 4 * q + (r16 >> 2), f7 = fr & 7;
  const int wn = (wave & 1) * (BN / 2), wk = (wave >> 1) * (BK / 2);
  auto join = [](v4s a, v4s b) { return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7)); };
  const uint32_t y_rd = uint32_t(fr * YROW + 8 * (r16 & 3));
  auto read_y = [&](uint32_t slot, int f) -> v8bf {
    lds_u8* at = (lds_u8*)lds + (slot * YB + y_rd + uint32_t(32 * ((wn / 16 + f) ^ f7)));
    return join(read_tr(at), read_tr(at + 16 * YROW));
  };
  const int x_plane = (r16 >> 1) & 1, x7 = f7 ^ x_plane;
  const uint32_t x_rd = uint32_t(X0 + fr * XROW + x_plane * (XROW / 2) + 8 * (r16 & 1));
  auto read_x = [&](uint32_t stage, int f) -> v8bf {
    lds_u8* at = (lds_u8*)lds + (stage * XB + x_rd + uint32_t(16 * ((wk / 16 + f) ^ x7)));
    return join(read_tr(at), read_tr(at + 16 * XROW));
  };

  v4f acc[KI][NI];
#pragma unroll
  for (int j = 0; j < KI; ++j)
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
  v8bf fx[KI], fy[NI];

  if constexpr (kSingleStage) {
    // (uniform: all waves of the workgroup take the same steps)
    for (int s = 0; s < steps; ++s) {
      copy_x(s, 0);
      copy_y(s, 0);
      wait_vmem();
      read_raw(0);
#pragma unroll
      for (int w = 0; w < 4; ++w) decode_word(w);
      write_x(0);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < KI; ++j) fx[j] = read_x(0, j);
#pragma unroll
      for (int i = 0; i < NI; ++i) fy[i] = read_y(0, i);
#pragma unroll
      for (int j = 0; j < KI; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[j], fy[i], acc[j][i], 0, 0, 0);
      __syncthreads();                            // the stage has been read
    }
  }

  // Step s multiplies the operands in registers and reads those of step s + 1
  // (whose stages the last barrier has closed) into the registers that the
  // products free; it decodes X of step s + 2 into the stage that step s used,
  // then copies X of step s + 5 and dY of step s + 3.  Past the last row
  // everything reads zeros.  The copies are counted by hand (G per step, X
  // before dY): a step's own stay in flight over its end, those of the step before
  // have landed there, X of step s + 4 with them, three steps before its use.
  constexpr int G = 2 + YC;
  // The first workgroups start 256 at a time, one per CU: of the two that share a
  // CU one goes first, so that one's stores overlap the other's products (8 experts
  // of 1024 rows, 4096 x 4096 FP32: 344 -> 332 us).  Later ones start where a place
  // is free, so two of a CU may have the same priority.
  if ((blockIdx.x >> 8) & 1) __builtin_amdgcn_s_setprio(1);
  if (!kSingleStage && steps > 0) {
    // X of steps 0 and 1 through registers, everything else of the first steps
    // behind it: one wait for memory before the first product.  (The compiler's
    // waits for these loads do not know of the copies behind them and wait for all.)
    u32x4 first[2];
    float first_s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(p.X + (size_t(r0) + size_t(t) * BR) * K + k0, int(step_size(x_size, t)));
      const __amdgpu_buffer_rsrc_t rs =
          buffer_rsrc(p.sX + (size_t(r0) + size_t(t) * BR) * Kb + k0 / 128, int(step_size(s_size, t)));
      first[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, int(x_lane), 0, 0));
      first_s[t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, int(s_lane), 0, 0));
    }
    copy_x(2, 2);
    copy_y(0, 0);
    copy_x(3, 0);
    copy_y(1, 1);
    copy_x(4, 1);
    copy_y(2, 2);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      xraw = first[t];
      xs = first_s[t];
#pragma unroll
      for (int w = 0; w < 4; ++w) decode_word(w);
      write_x(t);
    }
    wait_vmem_n<G>();                             // dY of steps 0 and 1, whatever the compiler waited for
    __syncthreads();
#pragma unroll
    for (int j = 0; j < KI; ++j) fx[j] = read_x(0, j);
#pragma unroll
    for (int i = 0; i < NI; ++i) fy[i] = read_y(0, i);
    __syncthreads();
    uint32_t a = 0, b = 1, c2 = 2;                // slots of steps s, s + 1, s + 2 (modulo 3)
    for (int s = 0; s < steps; ++s) {
      const uint32_t xst = (s + 1) & 1;
#pragma unroll
      for (int j = 0; j < KI; ++j) {
        if (j == 0) read_raw(c2);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[j], fy[i], acc[j][i], 0, 0, 0);
          if (j == KI - 1) fy[i] = read_y(b, i);
        }
        fx[j] = read_x(xst, j);
        if (j == 1 || j == 2) {
          decode_word(2 * j - 2);
          decode_word(2 * j - 1);
        }
        if (j == 2) write_x(s & 1);
        if (j == KI - 2) {
          copy_x(s + 5, c2);
          copy_y(s + 3, a);
        }
      }
      wait_vmem_n<G>();                           // all but X of step s + 5 and dY of s + 3
      __syncthreads();
      const uint32_t t = a;
      a = b;
      b = c2;
      c2 = t;
    }
    wait_vmem();                                  // no copy lands in LDS from here on
    __syncthreads();
  }

  // acc[j][i] of lane (q, r16) is row n0 + wn + 16 i + r16, columns
  // k0 + wk + 16 j + 4 q .. + 3.  Through LDS, 16 rows at a time in the wave's own
  // part (granules of 16 bytes at g ^ row), so that stores write whole lines.
  constexpr int GR = 4 * KI;                      // granules of a row
  constexpr int V = OUT_BF16 ? 8 : 4;             // columns of a 16-byte store
  constexpr int LR = 4 * GR / V;                  // lanes of a row
  v4f* part = reinterpret_cast<v4f*>(lds) + wave * 16 * GR;
  const int lrow = lane / LR, lcol = V * (lane % LR);
  const int k = k0 + wk + lcol;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int j = 0; j < KI; ++j) part[r16 * GR + ((4 * j + q) ^ r16 % GR)] = acc[j][i];
    __builtin_amdgcn_wave_barrier();              // a wave's LDS operations keep their order
#pragma unroll
    for (int h = 0; h < 16; h += 64 / LR) {
      const int row = lrow + h, n = n0 + wn + 16 * i + row;
      v4f v[V / 4];
#pragma unroll
      for (int c = 0; c < V / 4; ++c) v[c] = part[row * GR + ((lcol / 4 + c) ^ row % GR)];
      if (n < N && k < K) {
        const size_t at = (size_t(e) * N + n) * K + k;
        if constexpr (OUT_BF16) {
          u32x4_nt* dst = reinterpret_cast<u32x4_nt*>(static_cast<uint16_t*>(p.dW) + at);
          if (p.accumulate) {
            const u32x4_nt o = *dst;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              v[c / 2][2 * (c & 1)] += __uint_as_float(o[c] << 16);
              v[c / 2][2 * (c & 1) + 1] += __uint_as_float(o[c] & 0xFFFF0000u);
            }
          }
          store16<true>(dst, u32x4_nt{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]),
                                       pack_bf16x2(v[1][0], v[1][1]), pack_bf16x2(v[1][2], v[1][3])});
        } else {
          v4f* dst = reinterpret_cast<v4f*>(static_cast<float*>(p.dW) + at);
          if (p.accumulate) v[0] += *dst;
          store16<true>(dst, __builtin_bit_cast(u32x4_nt, v[0]));
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

#define DG_WGRAD_KERNEL_DEF(NAME, BN, BK, BF16) \
  __global__ __launch_bounds__(256, 2) void NAME(WgradArgs p) { wgrad_body<BN, BK, BF16>(p); }
#define DG_WGRAD_KERNEL_DECL(NAME, BN, BK, BF16) \
  __global__ __launch_bounds__(256, 2) void NAME(WgradArgs p);
DG_KERNEL(DG_WGRAD_KERNEL, WGRAD)(dg_wgrad256_bf16, 256, 128, true)
DG_KERNEL(DG_WGRAD_KERNEL, WGRAD)(dg_wgrad256_f32, 256, 128, false)
DG_KERNEL(DG_WGRAD_KERNEL, WGRAD)(dg_wgrad128_bf16, 128, 128, true)
DG_KERNEL(DG_WGRAD_KERNEL, WGRAD)(dg_wgrad128_f32, 128, 128, false)
#undef DG_WGRAD_KERNEL_DECL
#undef DG_WGRAD_KERNEL_DEF

}  // namespace dg
