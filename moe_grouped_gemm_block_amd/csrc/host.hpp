// Host side shared by the operators around the products: argument checks and launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dg.h"
#include "moe.hpp"

namespace dg_host {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// a row's bytes stay below 2^24, its pieces and blocks are counted in 32 bits
constexpr int64_t kMaxWidth = int64_t(1) << 22;
// slots are counted in 32 bits, a chunk past the last one included
constexpr int64_t kMaxSlots = int64_t(1) << 30;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// a pointer that has to be there, aligned
inline bool bad(const void* p, uintptr_t a) { return p == nullptr || !aligned(p, a); }
inline bool valid_type(int t) { return t == DG_IN_F32 || t == DG_IN_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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

}  // namespace dg_host
