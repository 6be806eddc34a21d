// Sums and maxima over groups of lanes, gfx950.
//
// A group is 16 lanes (one row of the lane permutations of vector instructions) or
// the whole wave.  Every lane gets the result, by butterflies in a fixed order, so
// that results do not depend on timing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace dg {

// v of the lane `ROR` before this one in its row of 16, cyclically
template <int ROR, typename T>
__device__ __forceinline__ T row_rotated(T v) {
  constexpr int CTRL = 0x120 + ROR;
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
  } else {
    const int2 b = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(T, make_int2(__builtin_amdgcn_mov_dpp(b.x, CTRL, 0xF, 0xF, true),
                                           __builtin_amdgcn_mov_dpp(b.y, CTRL, 0xF, 0xF, true)));
  }
}

// f(v, v of the lane 16 or 32 away), the same operand first in both lanes: one
// instruction exchanges rows (or halves) of two registers, both of them copies of v
template <int D>
__device__ __forceinline__ uint2 rows_exchanged(uint32_t v) {
  static_assert(D == 16 || D == 32, "rows or halves");
  if constexpr (D == 16) return __builtin_bit_cast(uint2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
  else return __builtin_bit_cast(uint2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
}
template <int D, typename T, typename F>
__device__ __forceinline__ T across(T v, F f) {
  if constexpr (sizeof(T) == 4) {
    const uint2 r = rows_exchanged<D>(__builtin_bit_cast(uint32_t, v));
    return f(__builtin_bit_cast(T, r.x), __builtin_bit_cast(T, r.y));
  } else {
    const uint2 b = __builtin_bit_cast(uint2, v);
    const uint2 x = rows_exchanged<D>(b.x), y = rows_exchanged<D>(b.y);
    return f(__builtin_bit_cast(T, make_uint2(x.x, y.x)), __builtin_bit_cast(T, make_uint2(x.y, y.y)));
  }
}

template <int L, typename T, typename F>
__device__ __forceinline__ T group_reduce(T v, F f) {
  static_assert(L == 16 || L == 64, "a row or a wave");
  v = f(v, row_rotated<8>(v));
  v = f(v, row_rotated<4>(v));
  v = f(v, row_rotated<2>(v));
  v = f(v, row_rotated<1>(v));
  if constexpr (L == 64) {
    v = across<16>(v, f);
    v = across<32>(v, f);
  }
  return v;
}

template <int L, typename T>
__device__ __forceinline__ T group_sum(T v) {
  return group_reduce<L>(v, [](T a, T b) { return a + b; });
}

template <int L, typename T>
__device__ __forceinline__ T group_max(T v) {
  return group_reduce<L>(v, [](T a, T b) { return a > b ? a : b; });
}

}  // namespace dg
