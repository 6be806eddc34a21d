// The global norm of many gradients, and their clipping, gfx950.
//
//   norm = sqrt(sum over all tensors of g^2);   out = g min(1, max_norm / norm)
//
// The tensors' addresses and sizes are arguments of the launch itself (up to
// kClipTensors a launch), so that nothing has to be laid out on the device first and a
// captured graph holds them.  Work is cut into chunks of kClipChunk elements, a
// workgroup each; a chunk finds its tensor by a binary search over the tensors' first
// chunks.  Squares are summed in 64 bits (FP32's largest gradients then do not
// overflow), the chunks' sums in their order: nothing is atomic.
//
// Bound by memory: 201 M BF16 gradients into FP32 66 us for the squares (6.1 TB/s), 4.8 for
// their sum and 191 for the scaling (6.3 TB/s).  The gradients are read twice, since the
// factor is known after the last of them; of few elements it is the two launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "groups.hpp"
#include "moe.hpp"

namespace dg {

constexpr int kClipTensors = 96;
constexpr int kClipThreads = 256;
constexpr int kClipChunk = 16384;

struct ClipTensor {
  const void* g;
  void* out;                 // clipping only
  int64_t n;
  int32_t first;             // first chunk
  uint8_t bf16, out_bf16, whole, pad;   // whole: 16-byte aligned
};

struct ClipBatch {
  ClipTensor t[kClipTensors];
  int count, chunks;
  double* part;              // [chunks], this launch's
  const float* norm;         // clipping
  float* norm_out;           // the norm of few elements
  float max_norm;
};
static_assert(sizeof(ClipBatch) <= 4096, "arguments of a launch");

__device__ __forceinline__ int clip_tensor(const ClipBatch& p, int chunk) {
  int lo = 0, hi = p.count - 1;                 // the last tensor whose first chunk is not past this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].first <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A thread's share of the squares of a chunk's n elements, kClipThreads threads together.
template <bool BF16>
__device__ __forceinline__ double chunk_squares(const ClipTensor& x, int64_t begin, int n, int thread) {
  constexpr int V = BF16 ? 8 : 4;
  double sum = 0.0;
  int done = 0;
  if (x.whole) {
    done = n / V * V;
#pragma unroll 4
    for (int i = thread * V; i < done; i += kClipThreads * V) {
      float v[V];
      load_values<BF16, V>(x.g, size_t(begin) + i, v);
#pragma unroll
      for (int k = 0; k < V; ++k) sum += double(v[k]) * v[k];
    }
  }
  for (int i = done + thread; i < n; i += kClipThreads) {
    float v;
    load_values<BF16, 1>(x.g, size_t(begin) + i, &v);
    sum += double(v) * v;
  }
  return sum;
}

// A wave's sum of a chunk's squares.
__device__ __forceinline__ double wave_squares(const ClipBatch& p, int chunk, int thread) {
  const ClipTensor& x = p.t[clip_tensor(p, chunk)];
  const int64_t begin = int64_t(chunk - x.first) * kClipChunk;
  const int n = int(min(x.n - begin, int64_t(kClipChunk)));
  return group_sum<64>(x.bf16 ? chunk_squares<true>(x, begin, n, thread) : chunk_squares<false>(x, begin, n, thread));
}

__device__ __forceinline__ void clip_squares_body(const ClipBatch& p) {
  __shared__ double sums[kClipThreads / 64];
  const int chunk = block_index();
  if (chunk >= p.chunks) return;
  const double s = wave_squares(p, chunk, threadIdx.x);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) p.part[chunk] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

struct ClipNormArgs {
  const double* part;        // [n]
  int64_t n;
  float* norm;
};

constexpr int kClipNormThreads = 1024;

__device__ __forceinline__ void clip_norm_of(double s, float* norm) {
  __shared__ double sums[kClipNormThreads / 64];
  s = group_sum<64>(s);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kClipNormThreads / 64; ++w) s += sums[w];
    *norm = float(sqrt(s));
  }
}

__device__ __forceinline__ void clip_norm_body(const ClipNormArgs& p) {
  double s = 0.0;
  // (eight loads on their way at a time)
  for (int64_t i0 = threadIdx.x; i0 < p.n; i0 += 8 * kClipNormThreads) {
    double v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i0 + k * kClipNormThreads < p.n ? p.part[i0 + k * kClipNormThreads] : 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += v[k];
  }
  clip_norm_of(s, p.norm);
}

// Few elements: one workgroup squares and sums in one launch, four chunks at a time.
constexpr int64_t kClipFew = 65536;

__device__ __forceinline__ void clip_norm_few_body(const ClipBatch& p) {
  double s = 0.0;
  for (int chunk = threadIdx.x / kClipThreads; chunk < p.chunks; chunk += kClipNormThreads / kClipThreads)
    s += wave_squares(p, chunk, threadIdx.x % kClipThreads);
  clip_norm_of((threadIdx.x & 63) == 0 ? s : 0.0, p.norm_out);
}

// The factor f 2^e: f in [0.5, 1) with the power of two apart where FP32's normal numbers do
// not hold it with room for the gradients, else f itself and e = 0.
struct ClipFactor {
  float f;
  int e;
  __device__ __forceinline__ float operator()(float g) const { return __builtin_ldexpf(g * f, e); }
};

template <bool IN, bool OUT>
__device__ __forceinline__ void chunk_scaled(const ClipTensor& x, int64_t begin, int n, ClipFactor f) {
  int done = 0;
  if (x.whole) {
    // pieces of 16 bytes of the wider type, so that a wave's stores are of whole lines
    constexpr int V = IN && OUT ? 8 : 4;
    done = n / V * V;
#pragma unroll 4
    for (int i = threadIdx.x * V; i < done; i += kClipThreads * V) {
      float v[V];
      if constexpr (IN && !OUT) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x.g) + begin + i);
        v[0] = __uint_as_float(w.x << 16);
        v[1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(w.y << 16);
        v[3] = __uint_as_float(w.y & 0xFFFF0000u);
      } else {
        load_values<IN, V>(x.g, size_t(begin) + i, v);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = f(v[k]);
      if constexpr (!IN && OUT)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(x.out) + begin + i) =
            uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      else
        store_values<OUT, V>(x.out, size_t(begin) + i, v);
    }
  }
  for (int i = done + threadIdx.x; i < n; i += kClipThreads) {
    float v;
    load_values<IN, 1>(x.g, size_t(begin) + i, &v);
    v = f(v);
    store_values<OUT, 1>(x.out, size_t(begin) + i, &v);
  }
}

// NaN as the norm makes every gradient NaN; an infinite one makes them 0 (and
// infinite gradients NaN), as the formula does.
__device__ __forceinline__ ClipFactor clip_factor(float norm, float max_norm) {
  const double f = double(max_norm) / double(norm);
  if (f >= 1.0) return ClipFactor{1.f, 0};
  const bool far = f < 0x1p-100;
  return ClipFactor{float(far ? __builtin_amdgcn_frexp_mant(f) : f), far ? __builtin_amdgcn_frexp_exp(f) : 0};
}

// Chunks from a launch's last on: what the norm read last is still in the caches (201 M BF16 in
// 48 tensors into FP32 191 us, from the first on 215).  Lists of several launches go through
// these in their order, each from its last chunk.
__device__ __forceinline__ void clip_scale_body(const ClipBatch& p) {
  const int chunk = p.chunks - 1 - int(block_index());
  if (chunk < 0) return;
  const ClipFactor f = clip_factor(*p.norm, p.max_norm);
  const ClipTensor& x = p.t[clip_tensor(p, chunk)];
  if (f.f == 1.f && x.g == x.out) return;       // in place, and nothing to change
  const int64_t begin = int64_t(chunk - x.first) * kClipChunk;
  const int n = int(min(x.n - begin, int64_t(kClipChunk)));
  if (x.bf16) {
    if (x.out_bf16) chunk_scaled<true, true>(x, begin, n, f);
    else chunk_scaled<true, false>(x, begin, n, f);
  } else {
    if (x.out_bf16) chunk_scaled<false, true>(x, begin, n, f);
    else chunk_scaled<false, false>(x, begin, n, f);
  }
}

}  // namespace dg
