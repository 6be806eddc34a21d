// Tokens sorted by expert and back, gfx950: the steps around the grouped
// products of a mixture-of-experts layer.
//
// A slot s = t * top_k + j is token t's j-th choice; ids[s] names its expert
// and is dropped when it lies outside [0, G).  The sorted matrix holds expert
// e's slots, in slot order, in rows [o_e, o_e + count_e) of a segment padded to
// `align` rows; row_slot maps a row to its slot (-1: padding), slot_row a slot
// to its row (-1: dropped).
//
//   sort         o_e, count_e, row_slot, slot_row from ids
//   permute      Y[r] = X[row_slot[r] / top_k], zeros in padding rows, as it is
//                or quantised to E4M3 with 1 x 128 scales
//   combine      out[t] = sum_j w[t][j] Y[slot_row[t][j]]
//   combine_bwd  dY[slot_row[t][j]] = w[t][j] dOut[t],
//                dw[t][j] = <dOut[t], Y[slot_row[t][j]]>
//
// All of them are bound by memory (or, for a few tokens, by the launch).  The
// kernels are token-major: a token's row is read once and written to its top_k
// rows, not once per sorted row, and no output row has two writers, so nothing
// is atomic and every sum has a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "quant.hpp"

namespace dg {

// ---- sort ---------------------------------------------------------------------
// A stable counting sort.  Sixteen waves of a workgroup take consecutive runs
// of its slots; each counts its run per expert in LDS, the counts become each
// wave's first rows by prefix sums over waves (and over the workgroups before,
// and over experts), and each wave then hands out rows 64 slots at a time: the
// rank of a slot among equal experts of its 64 comes from one ballot per bit of
// the expert's number, so ranks follow slot order whatever the timing.
// Up to kSortSingle slots one workgroup does all of it in one launch.  Above
// that a first launch counts every workgroup's chunk (and fills row_slot with
// -1), a second has each workgroup sum the counts of all (at most 128 chunks,
// read from L2) and place its own slots: 131072 slots of 256 experts 4.9 + 8.0 us,
// bound by that walk over 64 slots at a time, not by its 2 MB.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortMaxGroups = 1024;
constexpr int kSortSingle = 8192;

struct SortArgs {
  const void* ids;       // [n]
  int n;                 // slots
  int G, align, M;
  int chunk;             // slots per workgroup, a multiple of kSortThreads
  int nb;                // workgroups
  int32_t* offs;         // [G + 1]
  int32_t* counts;       // [G]
  int32_t* row_slot;     // [M]
  int32_t* slot_row;     // [n]
  int32_t* hist;         // [nb][G], unused by the single launch
};

// Expert of a slot, -1 when dropped.
template <typename ID>
__device__ __forceinline__ int slot_expert(const SortArgs& p, int s) {
  const ID v = static_cast<const ID*>(p.ids)[s];
  return v >= 0 && v < ID(p.G) ? int(v) : -1;
}

// (unsigned: one stride past n may lie past 2^31)
__device__ __forceinline__ void fill_rows(int32_t* dst, uint32_t n, uint32_t first, uint32_t stride) {
  for (uint32_t i = first; i < n; i += stride) dst[i] = -1;
}

template <typename ID>
__device__ __forceinline__ void sort_count_body(const SortArgs& p) {
  __shared__ int32_t hist[kSortMaxGroups];
  const int t = threadIdx.x;
  for (int e = t; e < p.G; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int s0 = blockIdx.x * p.chunk, s1 = min(p.n, s0 + p.chunk);
  for (int s = s0 + t; s < s1; s += kSortThreads) {
    const int e = slot_expert<ID>(p, s);
    if (e >= 0) atomicAdd(&hist[e], 1);          // integers: the order does not matter
  }
  fill_rows(p.row_slot, p.M, blockIdx.x * kSortThreads + t, p.nb * kSortThreads);
  __syncthreads();
  for (int e = t; e < p.G; e += kSortThreads) p.hist[size_t(blockIdx.x) * p.G + e] = hist[e];
}

template <typename ID, bool SINGLE>
__device__ __forceinline__ void sort_place_body(const SortArgs& p) {
  __shared__ int32_t first[kSortWaves * kSortMaxGroups];     // [wave][expert]: count, then next row
  __shared__ int32_t wave_sum[kSortWaves];
  __shared__ int2 sums[SINGLE ? 1 : kSortThreads];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int blk = SINGLE ? 0 : blockIdx.x;
  const int G = p.G;
  for (int i = t; i < kSortWaves * G; i += kSortThreads) first[i] = 0;
  if constexpr (SINGLE) fill_rows(p.row_slot, p.M, t, kSortThreads);
  __syncthreads();
  const int per = p.chunk / kSortWaves;                       // a multiple of 64
  const int s0 = blk * p.chunk + wave * per, s1 = min(p.n, s0 + per);
  int32_t* mine = first + wave * G;
  for (int s = s0 + lane; s < s1; s += 64) {
    const int e = slot_expert<ID>(p, s);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();

  // thread e: expert e's slots in this chunk before each wave, in all chunks,
  // and in the chunks before this one
  int total = 0, before = 0;
  if constexpr (!SINGLE) {
    // the chunks' counts, read by all threads: `parts` threads share an expert
    // (131072 slots, 256 experts: 7.7 us, against 8.7 with one thread each)
    const int width = G <= 64 ? 64 : 1 << (32 - __builtin_clz(G - 1)), parts = kSortThreads / width;
    const int e = t & (width - 1), part = t / width;
    if (e < G) {
#pragma unroll 16
      for (int b = part; b < p.nb; b += parts) {
        const int c = p.hist[size_t(b) * G + e];
        total += c;
        before += b < blk ? c : 0;
      }
    }
    sums[t] = make_int2(total, before);
    __syncthreads();
    total = before = 0;
    if (t < G) {
      for (int i = 0; i < parts; ++i) {
        total += sums[i * width + t].x;
        before += sums[i * width + t].y;
      }
    }
  }
  if (t < G) {
    int here = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = first[w * G + t];
      first[w * G + t] = here;
      here += c;
    }
    if constexpr (SINGLE) total = here;
  }
  // exclusive sum of the padded segments over experts
  const int seg = (total + p.align - 1) / p.align * p.align;
  int sum = seg;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(sum, o, 64);
    sum += lane >= o ? v : 0;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  int offset = sum - seg;
  for (int w = 0; w < wave; ++w) offset += wave_sum[w];
  if (t < G) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) first[w * G + t] += offset + before;
    if (blk == 0) {
      p.offs[t] = offset;
      p.counts[t] = total;
    }
  }
  if (blk == 0 && t == 0) p.offs[G] = p.M;       // the last segment takes the rows that are left
  __syncthreads();

  const int bits = 32 - __builtin_clz(G);
  for (int sb = s0; sb < s1; sb += 64) {
    const int s = sb + lane;
    const bool in = s < s1;
    const int e = in ? slot_expert<ID>(p, s) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    int row = -1;
    if (e >= 0) {
      const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      const int next = mine[e];
      row = next + rank;
      // the wave's lanes have all read `next` (one instruction) before the
      // lowest lane of each expert moves it on
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (rank == 0) mine[e] = next + __popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (row < p.M) p.row_slot[row] = s;
    }
    if (in) p.slot_row[s] = row;
  }
}

// ---- grids ------------------------------------------------------------------------
// A grid has below 2^32 work-items along x, which matrices past 8 GB reach (a
// thread per element at odd widths): more than 2^kGridBits workgroups are launched
// as rows of that many, the last row whole.
constexpr int kGridBits = 23;
__device__ __forceinline__ uint32_t block_index() { return (blockIdx.y << kGridBits) + blockIdx.x; }

// ---- rows of padding --------------------------------------------------------------
// Sixteen rows per wave; `zero(r)` is called by the whole wave for each row
// without a slot.
template <typename F>
__device__ __forceinline__ void each_padding_row(const int32_t* row_slot, int M, long long wave, F zero) {
  const int lane = threadIdx.x & 63;
  const long long r = wave * 16 + lane;
  uint64_t pad = __ballot(lane < 16 && r < M && row_slot[r < M ? r : 0] < 0);
  while (pad) {
    const int i = __builtin_ctzll(pad);
    pad &= pad - 1;
    zero(wave * 16 + i);
  }
}

__device__ __forceinline__ void zero_row_elems(void* Y, size_t row, int H, int elem) {
  const int lane = threadIdx.x & 63;
  char* base = static_cast<char*>(Y) + row * H * elem;
  if ((H * elem) % 16 == 0) {
    for (int c = lane; c < H * elem / 16; c += 64) reinterpret_cast<uint4*>(base)[c] = uint4{0u, 0u, 0u, 0u};
  } else if (elem == 2) {
    for (int c = lane; c < H; c += 64) reinterpret_cast<uint16_t*>(base)[c] = 0;
  } else {
    for (int c = lane; c < H; c += 64) reinterpret_cast<uint32_t*>(base)[c] = 0u;
  }
}

// Row and place of item (block_index() WIDTH + t) where a row has `per` items (per
// WIDTH below 2^31, t < WIDTH): two divisions in 32 bits; the one in 64 bits that
// this stands for takes over a hundred instructions, a fifth of the gated
// activation's.  Unsigned: the last workgroups' rows may lie past 2^31, behind the
// matrix.
template <int WIDTH>
__device__ __forceinline__ void row_and_place(int t, int per, uint32_t& row, int& place) {
  const uint32_t d = uint32_t(per), b = block_index(), q = b / d;
  const uint32_t x = (b - q * d) * WIDTH + uint32_t(t);
  const uint32_t y = x / d;
  row = q * WIDTH + y;
  place = int(x - y * d);
}

// ---- permute ----------------------------------------------------------------------
struct PermuteArgs {
  const void* X;             // [T][H]
  void* Y;                   // [M][H] values, or E4M3 codes
  float* S;                  // [M][Kb] scales (codes only)
  const int32_t* slot_row;   // [T][k]
  const int32_t* row_slot;   // [M]
  int T, k, M, H, Kb;
  int main_blocks;           // workgroups of the tokens; the rest take rows of padding
};

// Pieces of 16 bytes where 16 divides a row's size, else one element: a piece is
// loaded once and stored to the token's k rows.  (8192 tokens of 2 choices, BF16,
// H = 2048: 21.6 us; H = 2047, whose rows start at odd addresses: 54.)
template <int ELEM, bool WIDE>
__device__ __forceinline__ void permute_body(const PermuteArgs& p) {
  typedef typename std::conditional<WIDE, uint4, typename std::conditional<ELEM == 2, uint16_t, uint32_t>::type>::type V;
  if (int(block_index()) >= p.main_blocks) {
    each_padding_row(p.row_slot, p.M, (long long)(block_index() - p.main_blocks) * 4 + (threadIdx.x >> 6),
                     [&](long long r) { zero_row_elems(p.Y, size_t(r), p.H, ELEM); });
    return;
  }
  const int per = WIDE ? p.H * ELEM / 16 : p.H;               // pieces of a row
  uint32_t t;
  int c;
  row_and_place<256>(threadIdx.x, per, t, c);
  if (t >= uint32_t(p.T)) return;
  const V v = static_cast<const V*>(p.X)[size_t(t) * per + c];
  for (int j = 0; j < p.k; ++j) {
    const int row = p.slot_row[(long long)t * p.k + j];
    if (row >= 0 && row < p.M) static_cast<V*>(p.Y)[size_t(row) * per + c] = v;
  }
}

// Power-of-two block scale 2^e: the least that keeps amax within +-448 = 0.875
// 2^9, not below 2^-126 so that scale and reciprocal are normal numbers.
__device__ __forceinline__ int pow2_exponent(float amax) {
  const int e = __builtin_amdgcn_frexp_expf(amax) - (__builtin_amdgcn_frexp_mantf(amax) > 0.875f ? 8 : 9);
  return max(e, -126);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }   // |e| <= 126

// Sixteen values of one block -> codes.  A power-of-two scale moves values
// without rounding, so the hardware conversion (nearest even) is exact; any
// other scale goes through the bracketed encoder of quant.hpp.
struct Codes16 {
  uint32_t w[4];
};

template <bool POW2, typename F>
__device__ __forceinline__ Codes16 encode16(F value, float amax, float& s) {
  Codes16 c;
  if constexpr (POW2) {
    const int e = pow2_exponent(amax);
    const bool some = amax > 0.f;
    s = some ? pow2f(e) : 1.f;
    const float r = some ? pow2f(-e) : 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c.w[j] = hw_codes4(value(4 * j) * r, value(4 * j + 1) * r, value(4 * j + 2) * r, value(4 * j + 3) * r);
  } else {
    s = scale_of(amax);
    const ScaleNorm sn = scale_norm(s);
    const FastScale fs = fast_scale(sn);
    bool flag = !fs.ok;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c.w[j] = fast_codes4(value(4 * j), value(4 * j + 1), value(4 * j + 2), value(4 * j + 3), fs, flag);
    if (flag) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c.w[j] = exact_codes4(value(4 * j), value(4 * j + 1), value(4 * j + 2), value(4 * j + 3), sn);
    }
  }
  return c;
}

template <bool IN_BF16>
__device__ __forceinline__ void load_q16(Q1Buf<IN_BF16>& b, const void* X, size_t e0, bool in) {
  constexpr int N = IN_BF16 ? 2 : 4;
  const uint4* src = IN_BF16 ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(X) + e0)
                             : reinterpret_cast<const uint4*>(static_cast<const float*>(X) + e0);
  if (in) {
#pragma unroll
    for (int i = 0; i < N; ++i) b.w[i] = load16_nt(src + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) b.w[i] = uint4{0u, 0u, 0u, 0u};
  }
}

// An 8-lane group takes one 1 x 128 block (16 values per lane; H is a multiple
// of 16, so a lane holds 16 values or, past a partial last block, none),
// quantises it once and stores its codes, one whole 128-byte line, to each of
// the token's rows.  16384 tokens of 8 choices, H = 4096: 149 us, 825 MB at 5.5
// TB/s, which is what plain stores of 4 KB rows in this order reach (a copy of
// whole matrices: 5.3).
template <bool IN_BF16, bool POW2>
__device__ __forceinline__ void permute_fp8_body(const PermuteArgs& p) {
  const int lane = threadIdx.x & 63;
  uint8_t* Q = static_cast<uint8_t*>(p.Y);
  if (int(block_index()) >= p.main_blocks) {
    each_padding_row(p.row_slot, p.M, (long long)(block_index() - p.main_blocks) * 4 + (threadIdx.x >> 6),
                     [&](long long r) {
                       uint4* row = reinterpret_cast<uint4*>(Q + size_t(r) * p.H);
                       for (int c = lane; c < p.H / 16; c += 64) row[c] = uint4{0u, 0u, 0u, 0u};
                       for (int c = lane; c < p.Kb; c += 64) p.S[size_t(r) * p.Kb + c] = 1.f;
                     });
    return;
  }
  uint32_t t;
  int kb;
  row_and_place<32>(threadIdx.x >> 3, p.Kb, t, kb);
  const int col = kb * 128 + 16 * (lane & 7);
  const bool in = t < uint32_t(p.T) && col < p.H;
  Q1Buf<IN_BF16> b;
  load_q16(b, p.X, in ? size_t(t) * p.H + col : 0, in);
  // the first rows are looked up while X is on its way
  constexpr int J = 8;
  int rows[J];
  const int32_t* slot_row = p.slot_row + (t < uint32_t(p.T) ? (long long)t * p.k : 0);
#pragma unroll
  for (int j = 0; j < J; ++j) rows[j] = in && j < p.k ? slot_row[j] : -1;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, __builtin_fabsf(q1_value(b, i)));
  amax = group8_max(amax);
  float s;
  const Codes16 c = encode16<POW2>([&](int i) { return q1_value(b, i); }, amax, s);
  const u32x4_nt w{c.w[0], c.w[1], c.w[2], c.w[3]};
  __shared__ float scale[32];
  if ((lane & 7) == 0) scale[threadIdx.x >> 3] = s;
#pragma unroll
  for (int j = 0; j < J; ++j)
    if (rows[j] >= 0 && rows[j] < p.M) store16<true>(Q + size_t(rows[j]) * p.H + col, w);
  if (in) {
    for (int j = J; j < p.k; ++j) {
      const int row = slot_row[j];
      if (row >= 0 && row < p.M) store16<true>(Q + size_t(row) * p.H + col, w);
    }
  }
  // scales in whole lines: the workgroup's 32 blocks of each choice side by side
  __syncthreads();
  uint32_t t2;
  int kb2;
  row_and_place<32>(threadIdx.x & 31, p.Kb, t2, kb2);
  if (t2 >= uint32_t(p.T)) return;
  for (int j = threadIdx.x >> 5; j < p.k; j += 8) {
    const int row = p.slot_row[(long long)t2 * p.k + j];
    if (row >= 0 && row < p.M) p.S[size_t(row) * p.Kb + kb2] = scale[threadIdx.x & 31];
  }
}

// ---- combine ----------------------------------------------------------------------
struct CombineArgs {
  const void* Y;             // [M][H]
  const float* w;            // [T][k], or null: all ones
  const int32_t* slot_row;   // [T][k]
  void* out;                 // [T][H]
  int T, k, M, H;
};

// V values from 16-byte pieces (V = 8 BF16 or 4 FP32) or, where 16 does not divide a
// row's size, single elements (8192 x 2 rows of 2047 BF16: combine 76 us, gradient
// 84; of 2048: 19 and 39), NT: as
// non-temporal loads and stores of the pieces.  Measured on operands from HBM:
// non-temporal stores take the combine of 8192 x 2 rows of 2048 from 18.7 to 16.7
// us and the gradient of 4096 x 2 rows of 4096 from 36.9 to 32.8 us; such loads
// of Y as well 19.7 and 32.4 us, and 15.8 instead of 11.3 us for 1009 x 6 rows of
// 1408, whose ends share cache lines.
template <bool BF16, int V, bool NT = false>
__device__ __forceinline__ void load_values(const void* src, size_t e0, float* v) {
  if constexpr (V == 1) {
    v[0] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(src)[e0]) : static_cast<const float*>(src)[e0];
  } else if constexpr (BF16) {
    const uint16_t* at = static_cast<const uint16_t*>(src) + e0;
    const uint4 w = NT ? load16_nt(at) : *reinterpret_cast<const uint4*>(at);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    const float* at = static_cast<const float*>(src) + e0;
    const uint4 w = NT ? load16_nt(at) : *reinterpret_cast<const uint4*>(at);
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
}

template <bool BF16, int V>
__device__ __forceinline__ void store_values(void* dst, size_t e0, const float* v) {
  if constexpr (V == 1) {
    if constexpr (BF16) static_cast<uint16_t*>(dst)[e0] = uint16_t(bf16_bits(v[0]));
    else static_cast<float*>(dst)[e0] = v[0];
  } else if constexpr (BF16) {
    store16<true>(static_cast<uint16_t*>(dst) + e0,
                   u32x4_nt{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                            pack_bf16x2(v[6], v[7])});
  } else {
    store16<true>(static_cast<float*>(dst) + e0,
                   u32x4_nt{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
  }
}

// A thread takes V columns of one token and adds its k rows in the order of the
// choices, in FP32, rounded once.  Rows of dropped slots are not read.
template <bool BF16, int V>
__device__ __forceinline__ void combine_body(const CombineArgs& p) {
  uint32_t t;
  int c;
  row_and_place<256>(threadIdx.x, p.H / V, t, c);
  if (t >= uint32_t(p.T)) return;
  c *= V;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 2
  for (int j = 0; j < p.k; ++j) {
    const int row = p.slot_row[(long long)t * p.k + j];
    const float w = p.w ? p.w[(long long)t * p.k + j] : 1.f;
    if (row < 0 || row >= p.M) continue;
    float y[V];
    load_values<BF16, V>(p.Y, size_t(row) * p.H + c, y);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = __builtin_fmaf(w, y[v], acc[v]);
  }
  store_values<BF16, V>(p.out, size_t(t) * p.H + c, acc);
}

// ---- combine_bwd --------------------------------------------------------------------
struct CombineBwdArgs {
  const void* dOut;          // [T][H]
  const void* Y;             // [M][H]
  const float* w;            // [T][k]
  const int32_t* slot_row;   // [T][k]
  const int32_t* row_slot;   // [M]
  void* dY;                  // [M][H]
  float* dw;                 // [T][k]
  int T, k, M, H;
};

// A workgroup takes one token: dOut's row is read once per four choices (once
// for top_k <= 4), multiplied into dY's rows and dotted with Y's; the dot
// products are summed per thread, over the wave, then over waves in order.
template <bool BF16, int V>
__device__ __forceinline__ void combine_bwd_body(const CombineBwdArgs& p) {
  constexpr int J = 4;
  __shared__ float part[4][J];
  const int t = block_index();
  if (t >= p.T) {
    each_padding_row(p.row_slot, p.M, (long long)(t - p.T) * 4 + (threadIdx.x >> 6),
                     [&](long long r) { zero_row_elems(p.dY, size_t(r), p.H, BF16 ? 2 : 4); });
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = 0; j0 < p.k; j0 += J) {
    int row[J];
    float w[J], acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool in = j0 + j < p.k;
      row[j] = in ? p.slot_row[(long long)t * p.k + j0 + j] : -1;
      if (row[j] >= p.M) row[j] = -1;
      w[j] = in ? p.w[(long long)t * p.k + j0 + j] : 0.f;
      acc[j] = 0.f;
    }
    for (int c = threadIdx.x * V; c < p.H; c += 256 * V) {
      float d[V];
      load_values<BF16, V>(p.dOut, size_t(t) * p.H + c, d);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (row[j] < 0) continue;
        float y[V], o[V];
        load_values<BF16, V>(p.Y, size_t(row[j]) * p.H + c, y);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          acc[j] = __builtin_fmaf(d[v], y[v], acc[j]);
          o[v] = w[j] * d[v];
        }
        store_values<BF16, V>(p.dY, size_t(row[j]) * p.H + c, o);
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) acc[j] += __shfl_xor(acc[j], o, 64);
      if (lane == 0) part[wave][j] = acc[j];
    }
    __syncthreads();
    if (int(threadIdx.x) < J && j0 + int(threadIdx.x) < p.k) {
      const int j = threadIdx.x;
      p.dw[(long long)t * p.k + j0 + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
    }
    __syncthreads();
  }
}

}  // namespace dg
