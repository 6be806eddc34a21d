// The router of a mixture-of-experts layer, gfx950: each token's experts and their
// weights from the router's logits, the experts' load and the balance loss, and the
// gradient of the logits.
//
//   x = a token's logits [E]; an expert whose logit is -inf is closed
//   softmax   s = p = e^x / sum e^x
//   sigmoid   s = 1 / (1 + e^-x),  p = s / sum s
//   choice    the k largest x (with a bias: s + bias, compared in 64 bits), the
//             lower index first where they are equal; -inf is never chosen
//   weights   w_j = scale s_j, or scale s_j / (sum over the chosen s)
//   load      counts_e = tokens that chose e, P_e = sum over tokens p_e,
//             n = tokens with a choice
//   loss      E / (k n^2) sum_e counts_e P_e
//   gradient  of the weights and of p (counts are constants):
//             softmax  ds/dx = diag(p) - p p^T;  sigmoid  ds/dx = s (1 - s)
//
// Shares of scores are formed from scores divided by e^m, m the largest logit among
// them (softmax) or that and 0, whichever is less (sigmoid), so that no share is
// 0 / 0 where all scores underflow.
//
// A group of L lanes takes a token, V logits per lane in pieces of four, which lie side by
// side over the lanes: lane l's v-th is logit 4 L (v / 4) + 4 l + v % 4, so that loads and
// stores are of whole lines.
//
// The forward pass is bound by vector instructions, not by memory: 16384 tokens, 8 of 256
// experts, biased sigmoid in FP32 with the load, 14.7 us (1.2 TB/s, the vector units busy about
// 67 % of the time) and 5.4 for the sums over workgroups; 2 of 64, softmax in BF16, 8192 tokens,
// 4.8 + 3.1 us.  Of the 1106 that a wave of the large batch takes, counted in the assembly,
// about 280 are the choice (nine rounds of 16 keys a lane and a maximum over 16 lanes), 220 the
// scores, 200 the biased sums and their keys, 70 loads and the largest logit, 70 the weights, 20
// the sums of p, the rest what a workgroup does once.  Of one token it is the launch, 2.5 us.  The gradient of the large batch takes 12.5 us, 2.8 TB/s: a
// token's loads, arithmetic and stores wait for each other, and all tokens start together.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "common.hpp"
#include "groups.hpp"
#include "moe.hpp"

namespace dg {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxBlocks = 256;       // workgroups, each with its own partial sums

struct RouteArgs {
  const void* x;             // [T][E]
  const float* bias;         // [E], or null
  const uint8_t* mask;       // [T] (0: no token), or null: all ones
  int32_t* ids;              // [T][k]
  float* w;                  // [T][k]
  int32_t* counts;           // [E], or null: no load and no loss
  float* sums;               // [E]
  int32_t* routed;           // [1]
  float* loss;               // [1]
  float* part_sums;          // [nb][E]
  int32_t* part_counts;      // [nb][E]
  int32_t* part_routed;      // [nb]
  double* terms;             // [E] counts_e P_e
  int32_t* done;             // workgroups of the last step that have ended
  int T, E, k, nb;
  int sigmoid, renorm, bias_aligned;
  float scale;
};

// e^d for d <= 0, NaN for NaN: 2^h, h about d log2(e), and what d is more than h log(2) as a
// second term.  Within 2^-22 of it where it is a normal number of FP32 (d >= -87); below 2^-126
// it has few bits or is 0.
__device__ __forceinline__ float exp_nonpos(float d) {
  d = __builtin_elementwise_maximum(d, -150.f);
  constexpr float LN2 = 0.693147182464599609f, LN2_LO = -1.90465429995776e-9f;   // their sum is log(2)
  const float h = d * 1.44269504088896341f;
  const float more = __builtin_fmaf(h, -LN2_LO, __builtin_fmaf(h, -LN2, d));
  const float e = __builtin_amdgcn_exp2f(h);
  return __builtin_fmaf(e, more, e);
}

// s e^-min(m, 0) (sigmoid) or e^(x - m) (softmax) for a logit x <= m
__device__ __forceinline__ float shifted_score(float x, float m, bool sigmoid) {
  if (!sigmoid) return exp_nonpos(x - m);
  const float a = exp_nonpos(-__builtin_fabsf(x));
  const float num = m < 0.f ? exp_nonpos(x - m) : (x > 0.f ? 1.f : a);
  return num * __builtin_amdgcn_rcpf(1.f + a);
}

// The same for V logits, and with REST what one_minus_sigmoid gives (1 for softmax).
// The branches are the wave's, not an element's: with one at each element its exponential
// waits for the one before.
template <bool REST, int V>
__device__ __forceinline__ void shifted_scores(const float (&x)[V], float m, bool sigmoid, float (&s)[V],
                                               float (&rest)[REST ? V : 1]) {
  if (!sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = exp_nonpos(x[v] - m);
      if constexpr (REST) rest[v] = 1.f;
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float a = exp_nonpos(-__builtin_fabsf(x[v])), r = __builtin_amdgcn_rcpf(1.f + a);
    const bool up = x[v] > 0.f;
    s[v] = (up ? 1.f : a) * r;
    if constexpr (REST) rest[v] = (up ? a : 1.f) * r;
  }
  if (__ballot(m < 0.f)) {                          // tokens whose scores may underflow
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float r = __builtin_amdgcn_rcpf(1.f + exp_nonpos(-__builtin_fabsf(x[v])));
      s[v] = m < 0.f ? exp_nonpos(x[v] - m) * r : s[v];
    }
  }
}

// 1 - 1 / (1 + e^-x) without cancellation
__device__ __forceinline__ float one_minus_sigmoid(float x) {
  const float a = exp_nonpos(-__builtin_fabsf(x));
  return (x > 0.f ? a : 1.f) * __builtin_amdgcn_rcpf(1.f + a);
}

// Unsigned integers in the order of the values: 0 for -inf, from 1 on for numbers, NaN
// last; -0 as 0.
constexpr uint32_t kClosedKeys = 0x3FFu;          // room below the first number's key, see the choice
constexpr uint32_t kNaNKey = 0xFFFFFFFFu - kClosedKeys;
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t key = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  // less what -inf has, 0x7FFFFF, but not below 0
  return x != x ? kNaNKey : __builtin_elementwise_sub_sat(key, 0x7FFFFFu);
}
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t b = uint64_t(__double_as_longlong(x + 0.0));
  const uint64_t key = b ^ (uint64_t(int64_t(b) >> 63) | 0x8000000000000000ull);
  return x != x ? ~uint64_t(0) : x == -__builtin_inf() ? 0u : key;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  key = key > 0xFF000001u ? 0xFFFFFFFFu : key + 0x7FFFFFu;         // (+inf has 0xFF000001)
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* x, size_t i) {
  if constexpr (BF16) return __uint_as_float(uint32_t(static_cast<const uint16_t*>(x)[i]) << 16);
  else return static_cast<const float*>(x)[i];
}

// The key of the choice: an order key with its lowest bits replaced, moved up so that those
// of closed experts, and no others, are at most kClosedKeys.  ZEROS: -0 as 0.
template <uint32_t NUMBER, bool ZEROS>
__device__ __forceinline__ uint32_t packed_key(float x, uint32_t number) {
  static_assert(NUMBER <= kClosedKeys, "numbers of closed experts");
  const uint32_t b = __float_as_uint(ZEROS ? x + 0.f : x);
  const uint32_t key = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  return ((x != x ? 0xFFFFFFFFu : key - (0x7FFFFFu - kClosedKeys)) & ~NUMBER) | number;
}

// Logit of lane l's v-th value, and back.
template <int L>
__device__ __forceinline__ int expert_of(int l, int v) { return 4 * L * (v / 4) + 4 * l + v % 4; }
template <int L>
__device__ __forceinline__ int lane_of(int e) { return e / 4 % L; }
template <int L>
__device__ __forceinline__ int value_of(int e) { return e / (4 * L) * 4 + e % 4; }

// A lane's V values of a row of E, `none` past its end.  `whole`: rows of a multiple of
// four values, aligned to four.
template <bool BF16, int L, int V>
__device__ __forceinline__ void load_row(const void* x, size_t row, int l, int E, bool whole, float none,
                                         float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const int e = expert_of<L>(l, 4 * i);
    float* o = v + 4 * i;
    if (whole) {
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = none;
      if (e >= E) continue;
      if constexpr (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x) + row + e);
        o[0] = __uint_as_float(w.x << 16);
        o[1] = __uint_as_float(w.x & 0xFFFF0000u);
        o[2] = __uint_as_float(w.y << 16);
        o[3] = __uint_as_float(w.y & 0xFFFF0000u);
      } else {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + row + e);
        o[0] = w.x;
        o[1] = w.y;
        o[2] = w.z;
        o[3] = w.w;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float w = logit<BF16>(x, row + min(e + c, E - 1));
        o[c] = e + c < E ? w : none;
      }
    }
  }
}

// e^d for d <= 0 in 64 bits, a few roundings off: 2^n times the series of e^r, r the
// rest by n log(2).  A loop over coefficients in constant memory, since the choice has no
// registers left for them (as literals they are held across it, 40 of them).
__device__ __constant__ const double kInverse[15] = {0.0,     1.0 / 1, 1.0 / 2,  1.0 / 3,  1.0 / 4,  1.0 / 5,  1.0 / 6, 1.0 / 7,
                                                     1.0 / 8, 1.0 / 9, 1.0 / 10, 1.0 / 11, 1.0 / 12, 1.0 / 13, 1.0 / 14};
__device__ __forceinline__ double exp_nonpos(double d) {
  d = d < -800.0 ? -800.0 : d;
  constexpr double LN2 = 0x1.62e42fefap-1, LN2_LO = 0x1.cf79abc9e3b3ap-40;   // their sum is log(2), n LN2 exact
  const double n = __builtin_rint(d * 1.4426950408889634);
  const double r = __builtin_fma(n, -LN2_LO, __builtin_fma(n, -LN2, d));
  double e = 1.0;
#pragma unroll 1
  for (int k = 14; k >= 1; --k) e = __builtin_fma(e, r * kInverse[k], 1.0);
  return __builtin_ldexp(e, int(n));
}

// One of the registers by a variable index.  (Constants from the start: in a loop the
// compiler takes a[i] where i == v, and puts the array into memory for it.)
template <typename T, int... I>
__device__ __forceinline__ T pick_of(const T (&a)[sizeof...(I)], int i, std::integer_sequence<int, I...>) {
  T r = a[0];
  ((r = i == I ? a[I] : r), ...);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ T pick(const T (&a)[V], int i) {
  return pick_of(a, i, std::make_integer_sequence<int, V>{});
}

__device__ __forceinline__ void write_loss(const RouteArgs& p, int n, double term) {
  *p.routed = n;
  *p.loss = n ? float(term * p.E / (double(p.k) * n * n)) : 0.f;
}

// ---- choice -----------------------------------------------------------------------
// A value's order key with its lowest bits replaced by the expert's number, the lower
// number larger: the largest of a group names its expert, where a search for the index
// beside whole keys takes another 36 instructions a choice.  No key is taken out: keys
// minus the last one taken, as unsigned numbers, are in the same order, and those already
// taken lie below all others (key - g < 2^32 - g from g on, and at least that, by wrapping
// round, below it), so the next one is the largest again.  What the lost bits leave open is
// settled afterwards: the choices go on past the k-th until one is certainly smaller than
// the one before, and where two in a row were too close to tell, lane j computes the j-th
// one's whole key, and they are ranked by those.  BF16 logits lose nothing.  Where more than
// a lane each are too close (rows of equal logits) the choice is made again with whole keys
// throughout.
//
// With a bias a key is of an FP32 approximation of s + bias, and the whole key of s +
// bias in 64 bits.  A score is off by at most 2^-21 of itself (sigmoid) or 2^-18
// (softmax: the terms' 2^-22 and up to 22 roundings of their sum's 2^-24, and what x - m
// rounded to costs), none is larger than `most`, and the sum with the bias rounds once.
__device__ __forceinline__ float biased_tolerance(float largest, float most, bool sigmoid) {
  return (sigmoid ? 0x1p-19f : 0x1p-16f) * most + 0x1p-22f * __builtin_fabsf(largest);
}

template <bool BF16, int L, int V, bool BIASED>
__device__ __forceinline__ void route_body(const RouteArgs& p) {
  constexpr int PER_WAVE = 64 / L, PER_BLOCK = kRouteWaves * PER_WAVE;
  static_assert(kRouteThreads % (L * V) == 0 && PER_BLOCK % (kRouteThreads / (L * V)) == 0, "threads share experts evenly");
  constexpr uint32_t NUMBER = L * V - 1;            // bits of an expert's number
  constexpr bool WHOLE_KEYS = BF16 && !BIASED;      // all of a key is above them
  __shared__ int32_t count[L * V];
  __shared__ __attribute__((aligned(16))) float part[PER_BLOCK][L * V];     // a group's sums of p
  __shared__ int routed_of[kRouteWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & (L - 1), base = lane & ~(L - 1);
  const bool balance = p.counts != nullptr, sigmoid = p.sigmoid != 0, whole = p.E % 4 == 0;
  const float inf = __builtin_inff();
  if (balance) {
    for (int e = threadIdx.x; e < L * V; e += kRouteThreads) count[e] = 0;
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      *reinterpret_cast<float4*>(part[wave * PER_WAVE + lane / L] + expert_of<L>(l, 4 * i)) = float4{0.f, 0.f, 0.f, 0.f};
    if (blockIdx.x == 0 && threadIdx.x == 0 && gridDim.x > 1) *p.done = 0;
    __syncthreads();
  }
  int routed_sum = 0;

  // (all lanes run every turn: a group past the last token has no open expert)
  for (long long t0 = (long long)blockIdx.x * PER_BLOCK; t0 < p.T; t0 += (long long)p.nb * PER_BLOCK) {
    const long long t = t0 + wave * PER_WAVE + lane / L;
    const bool there = t < p.T && (p.mask == nullptr || p.mask[t] != 0);
    const size_t row = size_t(t) * p.E;
    // (not known to be the same every turn: comparisons with it are cheaper than kept)
    int E = p.E;
    asm volatile("" : "+s"(E));
    float x[V];
    if (there) {
      load_row<BF16, L, V>(p.x, row, l, E, whole, -inf, x);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = -inf;
    }
    // (NaN where one of them is NaN)
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = __builtin_elementwise_maximum(m, x[v]);
    m = group_reduce<L>(m, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
    const bool open = m != -inf;
    if (!open) m = 0.f;

    // scores of all experts (over e^min(m, 0) or e^m), where something needs them; they
    // are not kept in registers during the choice
    float s[V], none[1];
    float z = 1.f, r = 1.f;
    [[maybe_unused]] float f = 1.f;                 // what makes them scores
    if (BIASED || balance || (!p.renorm && !sigmoid)) {
      shifted_scores<false>(x, m, sigmoid, s, none);
      z = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) z += s[v];
      z = group_sum<L>(z);
      if (!open) z = 1.f;
      r = 1.f / z;
      if constexpr (BIASED) f = sigmoid ? exp_nonpos(fminf(m, 0.f)) : r;
    }
    uint32_t key[V];
    [[maybe_unused]] auto biased = [&](const float (&s)[V], float (&sum)[V]) {
      load_row<false, L, V>(p.bias, 0, l, E, whole && p.bias_aligned, 0.f, sum);
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] = x[v] == -inf ? -inf : __builtin_fmaf(s[v], f, sum[v]);
    };
    {
      float sum[V];
      if constexpr (BIASED) {
        if (__ballot(!(m < inf))) {                 // tokens with NaN scores: a bias of -inf closes those too
          load_row<false, L, V>(p.bias, 0, l, E, whole && p.bias_aligned, 0.f, sum);
#pragma unroll
          for (int v = 0; v < V; ++v) x[v] = !(m < inf) && sum[v] == -inf ? -inf : x[v];
        }
        biased(s, sum);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t number = NUMBER - uint32_t(expert_of<L>(l, v));
        // (-0 and 0 as sums with a bias are too close to tell anyway)
        if constexpr (BIASED) key[v] = packed_key<NUMBER, false>(sum[v], number);
        else key[v] = packed_key<NUMBER, true>(x[v], number);
      }
    }

    // lane j of the group takes choice j
    const float most = sigmoid ? 1.f : f;
    uint32_t mine = 0, last = 0;
    // (behind the open experts come closed ones, of which there are enough: more keys than
    // choices in all)
    auto choose = [&] {
      uint32_t best = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) best = max(best, key[v] - last);
      last += group_max<L>(best);
    };
    choose();
    if (l == 0) mine = last;
    const bool routed = last > kClosedKeys;         // a bias of -inf may have closed the open ones
    if (balance && routed) {                        // (scores of other rows may be NaN)
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        float4* at = reinterpret_cast<float4*>(part[wave * PER_WAVE + lane / L] + expert_of<L>(l, 4 * i));
        float4 sum = *at;
        sum.x = __builtin_fmaf(s[4 * i], r, sum.x);
        sum.y = __builtin_fmaf(s[4 * i + 1], r, sum.y);
        sum.z = __builtin_fmaf(s[4 * i + 2], r, sum.z);
        sum.w = __builtin_fmaf(s[4 * i + 3], r, sum.w);
        *at = sum;
      }
    }
    for (int j = 1; j < p.k; ++j) {
      choose();
      if (l == j) mine = last;
    }
    [[maybe_unused]] bool close = false, more = false;
    int n = p.k;                                    // choices that there are
    if constexpr (!WHOLE_KEYS) {
      // whether the second key, in order behind the first, may be of as large a value
      auto too_close = [&](uint32_t first, uint32_t second) {
        const uint32_t high = (second | NUMBER) - kClosedKeys, low = (first & ~NUMBER) - kClosedKeys;
        if constexpr (BIASED) return !(key_value(low) - key_value(high) > biased_tolerance(key_value(low), most, sigmoid));
        else return high >= low;
      };
      choose();                                     // the one behind the last
      uint32_t behind = L == 16 ? row_rotated<15>(mine) : __shfl(mine, (lane + 1) & 63, 64);
      if (l == p.k - 1) behind = last;
      const uint64_t pairs = (__ballot(l < p.k && behind > kClosedKeys && too_close(mine, behind)) >> base) &
                             (L == 64 ? ~uint64_t(0) : uint64_t(0xFFFF));
      close = pairs != 0;
      more = (pairs >> (p.k - 1)) & 1;
      while (__ballot(more) && n < L) {
        if (l == n) mine = last;
        ++n;
        const uint32_t before = last;
        choose();
        more = last > kClosedKeys && too_close(before, last);
      }
    }
    int id = mine > kClosedKeys ? int(NUMBER - (mine & NUMBER)) : -1;

    if constexpr (!WHOLE_KEYS) {
      // s + bias in 64 bits
      double z64 = 1.0;
      [[maybe_unused]] auto all64 = [&] {
        if (sigmoid) return;
        z64 = 0.0;
#pragma unroll 1
        for (int v = 0; v < V; ++v) z64 += exp_nonpos(double(pick(x, v)) - double(m));
        z64 = group_sum<L>(z64);
      };
      [[maybe_unused]] auto sum64 = [&](float xv, float bias) {
        const double e = exp_nonpos(sigmoid ? -__builtin_fabs(double(xv)) : double(xv) - double(m));
        return (sigmoid && xv > 0.f ? 1.0 : e) / (sigmoid ? 1.0 + e : z64) + double(bias);
      };
      if (__ballot(close) && !__ballot(more)) {
        // the n choices ranked by their whole keys, equal ones by their numbers; lanes
        // without a choice behind them
        uint64_t kd = 0;
        if constexpr (BIASED) all64();
        if (l < n && id >= 0) {
          const float xv = logit<BF16>(p.x, row + id);
          if constexpr (BIASED) kd = order_key(sum64(xv, p.bias[id]));
          else kd = order_key(xv);
        }
        const int number = l < n && id >= 0 ? id : int(NUMBER) + 1 + l;
        int rank = 0;
        for (int i = 0; i < n; ++i) {
          const uint64_t ki = __shfl(kd, base + i, 64);
          const int ni = __shfl(number, base + i, 64);
          rank += ki > kd || (ki == kd && ni < number);
        }
        if (l >= n) rank = l;
        id = __builtin_amdgcn_ds_permute((base + rank) << 2, id);
      } else if (__ballot(close)) {
        // whole keys throughout
        if constexpr (BIASED) {
          float s[V], sum[V], none[1];
          shifted_scores<false>(x, m, sigmoid, s, none);
          biased(s, sum);
#pragma unroll
          for (int v = 0; v < V; ++v) key[v] = order_key(sum[v]);
          all64();
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) key[v] = order_key(x[v]);
        }
        id = -1;
#pragma unroll 1
        for (int j = 0; j < p.k; ++j) {
          uint32_t best = 0;
#pragma unroll
          for (int v = 0; v < V; ++v) best = max(best, key[v]);
          const uint32_t g = group_max<L>(best);
          // the lane's first of the largest
          int e = INT32_MAX;
          if constexpr (BIASED) {
            const float cut = key_value(g) - biased_tolerance(key_value(g), most, sigmoid);
            uint32_t near = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) near |= uint32_t(key[v] != 0 && !(key_value(key[v]) < cut)) << v;
            uint64_t kd = 0;
            float x_of = 0.f, bias_of = 0.f;        // what kd is of: the same again changes nothing
            while (__ballot(near != 0)) {
              const int v = near ? __builtin_ctz(near) : 0;
              const int ev = expert_of<L>(l, v);
              const float xv = pick(x, v), bv = p.bias[near ? ev : 0];
              const bool other = near != 0 && !(kd != 0 && xv == x_of && bv == bias_of);
              if (__ballot(other)) {
                const uint64_t kv = order_key(sum64(xv, bv));
                if (other && kv > kd) {
                  kd = kv;
                  e = ev;
                  x_of = xv;
                  bias_of = bv;
                }
              }
              near &= near - 1;
            }
            if (kd != group_max<L>(kd)) e = INT32_MAX;
          } else {
#pragma unroll
            for (int v = V - 1; v >= 0; --v) e = key[v] == g ? expert_of<L>(l, v) : e;
          }
          e = group_reduce<L>(e, [](int a, int b) { return a < b ? a : b; });
          if (l == j && g != 0) id = e;
#pragma unroll
          for (int v = 0; v < V; ++v) key[v] = expert_of<L>(l, v) == e ? 0u : key[v];
        }
      }
    }
    if (l >= p.k) id = -1;
    routed_sum += routed && l == 0;

    // weights, from the choices' logits (in the caches still)
    const float xs = id >= 0 ? logit<BF16>(p.x, row + id) : -inf;
    float w = 0.f;
    if (p.renorm) {
      uint32_t tc = order_key(xs);
      tc = group_max<L>(tc);
      const float mc = tc ? key_value(tc) : 0.f;
      const float s = id >= 0 ? shifted_score(xs, mc, sigmoid) : 0.f;
      const float sum = group_sum<L>(s);
      w = id >= 0 ? p.scale * (s / sum) : 0.f;
      // (NaN among a token's scores makes all of them NaN, but a bias may choose other experts)
      if (BIASED && !sigmoid && id >= 0 && !(m < inf)) w = __builtin_nanf("");
    } else if (id >= 0) {
      w = p.scale * (sigmoid ? shifted_score(xs, 0.f, true) : shifted_score(xs, m, false) / z);
    }
    if (l < p.k && t < p.T) {
      p.ids[t * p.k + l] = id;
      p.w[t * p.k + l] = w;
    }
    if (balance && id >= 0) atomicAdd(&count[id], 1);      // integers: the order does not matter
  }

  if (!balance) return;
  // over groups, in their order: threads that share an expert are a multiple of 64 apart
  routed_sum = group_sum<64>(routed_sum);
  if (lane == 0) routed_of[wave] = routed_sum;
  __syncthreads();
  constexpr int SHARE = kRouteThreads / (L * V), EACH = PER_BLOCK / SHARE;
  const int e = threadIdx.x % (L * V), share = threadIdx.x / (L * V);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < EACH; ++i) sum += part[share * EACH + i][e];
  __syncthreads();
  part[share][e] = sum;
  __syncthreads();
  const bool alone = gridDim.x == 1;               // then these are the sums
  double term = 0.0;
  if (share == 0 && e < p.E) {
#pragma unroll
    for (int i = 1; i < SHARE; ++i) sum += part[i][e];
    (alone ? p.sums : p.part_sums + size_t(blockIdx.x) * p.E)[e] = sum;
    (alone ? p.counts : p.part_counts + size_t(blockIdx.x) * p.E)[e] = count[e];
    term = double(sum) * count[e];
  }
  int n = 0;
  for (int w = 0; w < kRouteWaves; ++w) n += routed_of[w];
  if (!alone) {
    if (threadIdx.x == 0) p.part_routed[blockIdx.x] = n;
    return;
  }
  __shared__ double terms[kRouteWaves];
  term = group_sum<64>(term);
  if (lane == 0) terms[wave] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kRouteWaves; ++w) term += terms[w];
    write_loss(p, n, term);
  }
}

// The partial sums of all workgroups added up in their order, 32 experts a workgroup and
// 32 threads an expert, and by the workgroup that ends last the loss, in 64 bits.
// (Which one that is does not show: it adds the experts' terms in their order.)
constexpr int kFinishExperts = 32;
constexpr int kFinishParts = 32;

__device__ __forceinline__ void route_finish_body(const RouteArgs& p) {
  __shared__ float sums[kFinishParts][kFinishExperts + 1];
  __shared__ int32_t counts[kFinishParts][kFinishExperts + 1];
  const int col = threadIdx.x % kFinishExperts, part = threadIdx.x / kFinishExperts;
  const int e = blockIdx.x * kFinishExperts + col;
  float sum = 0.f;
  int count = 0;
  if (e < p.E) {
    // (at most kRouteMaxBlocks: all loads on their way at once)
    constexpr int N = kRouteMaxBlocks / kFinishParts;
    float s[N];
    int32_t c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int b = part + i * kFinishParts;
      s[i] = b < p.nb ? p.part_sums[size_t(b) * p.E + e] : 0.f;
      c[i] = b < p.nb ? p.part_counts[size_t(b) * p.E + e] : 0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      sum += s[i];
      count += c[i];
    }
  }
  // (for the workgroup that ends last, on their way early)
  int n = 0;
  if (threadIdx.x < 64)
    for (int b = threadIdx.x; b < p.nb; b += 64) n += p.part_routed[b];
  sums[part][col] = sum;
  counts[part][col] = count;
  __syncthreads();
  if (threadIdx.x >= 64) return;                   // the rest is one wave's
  if (part == 0 && e < p.E) {
#pragma unroll
    for (int i = 1; i < kFinishParts; ++i) {
      sum += sums[i][col];
      count += counts[i][col];
    }
    p.sums[e] = sum;
    p.counts[e] = count;
    p.terms[e] = double(sum) * count;
  }
  __threadfence();
  int ended = 0;
  if (threadIdx.x == 0) ended = atomicAdd(p.done, 1);
  if (__builtin_amdgcn_readfirstlane(ended) != int(gridDim.x) - 1) return;
  __threadfence();
  // (all loads on their way at once)
  double terms[kRouteMaxExperts / 64], term = 0.0;
#pragma unroll
  for (int i = 0; i < kRouteMaxExperts / 64; ++i) {
    const int at = threadIdx.x + 64 * i;
    terms[i] = at < p.E ? __hip_atomic_load(&p.terms[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
  }
#pragma unroll
  for (int i = 0; i < kRouteMaxExperts / 64; ++i) term += terms[i];
  term = group_sum<64>(term);
  n = group_sum<64>(n);
  if (threadIdx.x == 0) write_loss(p, n, term);
}

// The same by one workgroup, where there is little to add up: no other's terms to wait for
// (128 workgroups' sums of 64 experts: 3 us instead of 4.4).  Threads that share an expert
// are a power of two apart.
constexpr int kFinishOne = 16384;                  // partial sums up to which it is used

__device__ __forceinline__ void route_finish_one_body(const RouteArgs& p) {
  constexpr int THREADS = kFinishExperts * kFinishParts;
  __shared__ float sums[THREADS];
  __shared__ int32_t counts[THREADS];
  __shared__ double terms[THREADS / 64];
  __shared__ int ns[THREADS / 64];
  const int width = p.E <= 64 ? 64 : 1 << (32 - __builtin_clz(p.E - 1)), parts = THREADS / width;
  const int e = threadIdx.x & (width - 1), part = threadIdx.x / width;
  float sum = 0.f;
  int count = 0;
  if (e < p.E) {
    // (eight loads of each on their way at a time)
    for (int b0 = part; b0 < p.nb; b0 += 8 * parts) {
      float s[8];
      int32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int b = b0 + i * parts;
        s[i] = b < p.nb ? p.part_sums[size_t(b) * p.E + e] : 0.f;
        c[i] = b < p.nb ? p.part_counts[size_t(b) * p.E + e] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum += s[i];
        count += c[i];
      }
    }
  }
  int n = int(threadIdx.x) < p.nb ? p.part_routed[threadIdx.x] : 0;
  sums[threadIdx.x] = sum;
  counts[threadIdx.x] = count;
  __syncthreads();
  double term = 0.0;
  if (part == 0 && e < p.E) {
    for (int i = 1; i < parts; ++i) {
      sum += sums[i * width + e];
      count += counts[i * width + e];
    }
    p.sums[e] = sum;
    p.counts[e] = count;
    term = double(sum) * count;
  }
  term = group_sum<64>(term);
  n = group_sum<64>(n);
  if ((threadIdx.x & 63) == 0) {
    terms[threadIdx.x >> 6] = term;
    ns[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < THREADS / 64; ++w) {
      term += terms[w];
      n += ns[w];
    }
    write_loss(p, n, term);
  }
}

// ---- gradient ----------------------------------------------------------------------
struct RouteBwdArgs {
  const void* x;             // [T][E]
  const int32_t* ids;        // [T][k]
  const float* dw;           // [T][k]
  const int32_t* counts;     // [E], or null: no gradient of the loss
  const int32_t* routed;     // [1]
  const float* dloss;        // [1]
  void* dx;                  // [T][E]
  int T, E, k;
  int sigmoid, renorm, counts_aligned;
  float scale;
};

constexpr int kRouteBwdThreads = 256;

// dx = sum over choices of u_j at their experts, plus p times what the loss and, for
// softmax, the other scores take off:
//   shares q_j       u_j = scale q_j (dw_j - sum_i q_i dw_i) [(1 - s_j) for sigmoid]
//   softmax, plain   u_j = scale p_j dw_j, and - p_e sum_j u_j at every expert
//   sigmoid, plain   u_j = scale s_j (1 - s_j) dw_j
//   loss             f_e = dloss E / (k n^2) counts_e: p_e (f_e - sum p f) [(1 - s_e)]
// A token without choices adds nothing, whatever its logits are.  An expert that a token
// names twice gets both gradients, in their order.  The u_j reach their experts' lanes
// through LDS.
template <bool BF16, int L, int V>
__device__ __forceinline__ void route_bwd_body(const RouteBwdArgs& p) {
  constexpr int PER_BLOCK = kRouteBwdThreads / L;
  __shared__ __attribute__((aligned(16))) float at_expert[PER_BLOCK][L * V];
  const int lane = threadIdx.x & 63;
  const int l = lane & (L - 1), base = lane & ~(L - 1);
  const bool sigmoid = p.sigmoid != 0, whole = p.E % 4 == 0, loss = p.counts != nullptr;
  const long long t = (long long)block_index() * PER_BLOCK + threadIdx.x / L;
  const bool in = t < p.T;
  const size_t row = size_t(t) * p.E;
  const float inf = __builtin_inff();
  const bool all = loss || !(p.renorm || sigmoid);
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = -inf;
  if (all && in) load_row<BF16, L, V>(p.x, row, l, p.E, whole, -inf, x);
  int id = in && l < p.k ? p.ids[t * p.k + l] : -1;
  if (id >= p.E) id = -1;
  const uint64_t any = __ballot(id >= 0) >> base;
  const bool routed = (L == 64 ? any : any & 0xFFFFu) != 0;
  float xs = -inf;
  const float dw = id >= 0 ? p.scale * p.dw[t * p.k + l] : 0.f;
  // (a wave reads and writes its own tokens' rows only)
  float* mine = at_expert[threadIdx.x / L];

  // what every expert gets: p_e (f_e - off), for sigmoid times 1 - s_e
  float pe[V], f[V], rest[V], off = 0.f, z = 1.f, m = 0.f;
  if (!all) {
    if (id >= 0) xs = logit<BF16>(p.x, row + id);
  } else {
    // the choices' logits come through LDS, not by another read that waits for the ids
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      *reinterpret_cast<float4*>(mine + expert_of<L>(l, 4 * i)) = float4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (id >= 0) xs = mine[id];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = routed ? x[v] : -inf;
    m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = __builtin_elementwise_maximum(m, x[v]);
    m = group_reduce<L>(m, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
    const bool open = m != -inf;
    if (!open) m = 0.f;
    shifted_scores<true>(x, m, sigmoid, pe, rest);
    z = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) z += pe[v];
    z = group_sum<L>(z);
    if (!open) z = 1.f;
    const float r = 1.f / z;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      pe[v] *= r;
      f[v] = 0.f;
    }
    if (loss) {
      const double n = *p.routed;
      const float c = n > 0.0 ? float(double(*p.dloss) * p.E / (double(p.k) * n * n)) : 0.f;
      load_row<false, L, V>(p.counts, 0, l, p.E, whole && p.counts_aligned, 0.f, f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f[v] = c * float(__float_as_int(f[v]));
        off = __builtin_fmaf(pe[v], f[v], off);
      }
      off = group_sum<L>(off);
    }
  }

  float u = 0.f;
  if (p.renorm) {
    uint32_t tc = order_key(xs);
    tc = group_max<L>(tc);
    const float mc = tc ? key_value(tc) : 0.f;
    const float s = id >= 0 ? shifted_score(xs, mc, sigmoid) : 0.f;
    const float sum = group_sum<L>(s);
    const float q = tc && id >= 0 ? s / sum : 0.f;
    const float mean = group_sum<L>(q * dw);
    u = q * (dw - mean);
    if (sigmoid) u *= one_minus_sigmoid(xs);
  } else if (id >= 0) {
    if (sigmoid) {
      u = dw * shifted_score(xs, 0.f, true) * one_minus_sigmoid(xs);
    } else {
      u = dw * (shifted_score(xs, m, false) / z);
    }
  }
  if (!p.renorm && !sigmoid) off += group_sum<L>(u);

#pragma unroll
  for (int i = 0; i < V / 4; ++i) *reinterpret_cast<float4*>(mine + expert_of<L>(l, 4 * i)) = float4{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  bool twice = false;
  for (int j = 0; j < p.k - 1; ++j) {
    const int other = __shfl(id, base + j, 64);     // (by all lanes: the source takes part)
    twice = twice || (l > j && id >= 0 && id == other);
  }
  if (!__ballot(twice)) {
    if (id >= 0) mine[id] = u;
  } else {
    for (int j = 0; j < p.k; ++j) {
      if (l == j && id >= 0) mine[id] += u;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (!in) return;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const int e = expert_of<L>(l, 4 * i);
    if (e >= p.E) continue;
    const float4 w = *reinterpret_cast<const float4*>(mine + e);
    float d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (all) d[c] += pe[4 * i + c] * (f[4 * i + c] - off) * rest[4 * i + c];
      if (!routed) d[c] = 0.f;
    }
    if (whole) {
      if constexpr (BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dx) + row + e) =
            uint2{pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3])};
      else *reinterpret_cast<float4*>(static_cast<float*>(p.dx) + row + e) = float4{d[0], d[1], d[2], d[3]};
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (e + c >= p.E) continue;
        if constexpr (BF16) static_cast<uint16_t*>(p.dx)[row + e + c] = uint16_t(bf16_bits(d[c]));
        else static_cast<float*>(p.dx)[row + e + c] = d[c];
      }
    }
  }
}

}  // namespace dg
