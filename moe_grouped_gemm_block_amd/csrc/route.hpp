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
// A group of L lanes takes a token, V logits per lane, lane l those from l V on: the
// lowest lane that holds the largest value then also holds the lowest index.
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
  int T, E, k, nb;
  int sigmoid, renorm;
  float scale;
};

// e^d for d <= 0 within 2^-22 of it, 0 below -104, NaN for NaN (the product with
// log2(e) keeps its rounding error as a second term)
__device__ __forceinline__ float exp_nonpos(float d) {
  d = d < -150.f ? -150.f : d;
  constexpr float L2E = 1.44269504088896341f, L2E_LO = 1.92596299e-8f;   // their sum is log2(e)
  const float hi = d * L2E;
  const float lo = __builtin_fmaf(d, L2E, -hi) + d * L2E_LO;
  const float e = __builtin_amdgcn_exp2f(hi);
  return __builtin_fmaf(e, lo * 0.693147180559945f, e);
}

// s e^-min(m, 0) (sigmoid) or e^(x - m) (softmax) for a logit x <= m
__device__ __forceinline__ float shifted_score(float x, float m, bool sigmoid) {
  if (!sigmoid) return exp_nonpos(x - m);
  const float a = exp_nonpos(-__builtin_fabsf(x));
  const float num = m < 0.f ? exp_nonpos(x - m) : (x > 0.f ? 1.f : a);
  return num * __builtin_amdgcn_rcpf(1.f + a);
}

// 1 - 1 / (1 + e^-x) without cancellation
__device__ __forceinline__ float one_minus_sigmoid(float x) {
  const float a = exp_nonpos(-__builtin_fabsf(x));
  return (x > 0.f ? a : 1.f) * __builtin_amdgcn_rcpf(1.f + a);
}

// Unsigned integers in the order of the values: 0 for -inf, NaN last, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t key = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  return x != x ? 0xFFFFFFFFu : x == -__builtin_inff() ? 0u : key;
}
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t b = uint64_t(__double_as_longlong(x + 0.0));
  const uint64_t key = b ^ (uint64_t(int64_t(b) >> 63) | 0x8000000000000000ull);
  return x != x ? ~uint64_t(0) : x == -__builtin_inf() ? 0u : key;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// V logits from element e0 of a row on, -inf past its end.  `whole`: rows of a
// multiple of V logits, which then lie in or out together.
template <bool BF16, int V>
__device__ __forceinline__ void load_logits(const void* x, size_t row, int e0, int E, bool whole, float (&v)[V]) {
  if (whole && e0 < E) {
    if constexpr (BF16) {
      const uint16_t* src = static_cast<const uint16_t*>(x) + row + e0;
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const uint2 w = reinterpret_cast<const uint2*>(src)[i];
        v[4 * i] = __uint_as_float(w.x << 16);
        v[4 * i + 1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[4 * i + 2] = __uint_as_float(w.y << 16);
        v[4 * i + 3] = __uint_as_float(w.y & 0xFFFF0000u);
      }
    } else {
      const float* src = static_cast<const float*>(x) + row + e0;
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 w = reinterpret_cast<const float4*>(src)[i];
        v[4 * i] = w.x;
        v[4 * i + 1] = w.y;
        v[4 * i + 2] = w.z;
        v[4 * i + 3] = w.w;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = -__builtin_inff();
    if (e0 + i < E) {
      if constexpr (BF16) v[i] = __uint_as_float(uint32_t(static_cast<const uint16_t*>(x)[row + e0 + i]) << 16);
      else v[i] = static_cast<const float*>(x)[row + e0 + i];
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

// Choices by score + bias.  The sums are compared in FP32 first: a score is off by at
// most 2^-21 of itself (sigmoid), or 2^-18 (softmax: the terms' 2^-22 and up to 22
// roundings of their sum's 2^-24, and of e^(x - m) what x - m rounded to costs), and
// none is larger than `most`; the sum with the bias rounds once.  Where two sums that
// follow each other are closer than twice that, the choice is made again with those that
// are that close to the largest compared in 64 bits.
__device__ __forceinline__ float biased_tolerance(float largest, float most, bool sigmoid) {
  return (sigmoid ? 0x1p-19f : 0x1p-16f) * most + 0x1p-22f * __builtin_fabsf(largest);
}

// One workgroup of kRouteThreads: the partial sums of all workgroups added up in
// their order, and the loss in 64 bits.
__device__ __forceinline__ void route_finish(const RouteArgs& p) {
  __shared__ double terms[kRouteWaves];
  __shared__ int ns[kRouteWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  double term = 0.0;
  for (int e = t; e < p.E; e += kRouteThreads) {
    float sum = 0.f;
    int count = 0;
    for (int b = 0; b < p.nb; ++b) {
      sum += p.part_sums[size_t(b) * p.E + e];
      count += p.part_counts[size_t(b) * p.E + e];
    }
    p.sums[e] = sum;
    p.counts[e] = count;
    term += double(sum) * count;
  }
  int n = 0;
  for (int b = t; b < p.nb; b += kRouteThreads) n += p.part_routed[b];
  term = group_sum<64>(term);
  n = group_sum<64>(n);
  if (lane == 0) {
    terms[wave] = term;
    ns[wave] = n;
  }
  __syncthreads();
  if (t == 0) {
    for (int w = 1; w < kRouteWaves; ++w) {
      term += terms[w];
      n += ns[w];
    }
    *p.routed = n;
    *p.loss = n ? float(term * p.E / (double(p.k) * n * n)) : 0.f;
  }
}

template <bool BF16, int L, int V, bool BIASED>
__device__ __forceinline__ void route_body(const RouteArgs& p) {
  constexpr int PER_WAVE = 64 / L, PER_BLOCK = kRouteWaves * PER_WAVE;
  __shared__ int32_t count[L * V];
  __shared__ float part[kRouteWaves][L * V];             // expert l V + v at v L + l: no bank conflicts
  __shared__ int routed_of[kRouteWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & (L - 1), base = lane & ~(L - 1);
  const int e0 = l * V;
  const bool balance = p.counts != nullptr, sigmoid = p.sigmoid != 0, whole = p.E % V == 0;
  if (balance) {
    for (int e = threadIdx.x; e < L * V; e += kRouteThreads) count[e] = 0;
    for (int i = lane; i < L * V; i += 64) part[wave][i] = 0.f;     // (the wave's own)
    __syncthreads();
  }
  int routed_sum = 0;

  // (all lanes run every turn: a group past the last token has no open expert)
  for (long long t0 = (long long)blockIdx.x * PER_BLOCK; t0 < p.T; t0 += (long long)p.nb * PER_BLOCK) {
    const long long t = t0 + wave * PER_WAVE + lane / L;
    const bool there = t < p.T && (p.mask == nullptr || p.mask[t] != 0);
    float x[V];
    if (there) {
      load_logits<BF16, V>(p.x, size_t(t) * p.E, e0, p.E, whole, x);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = -__builtin_inff();
    }
    uint32_t key[V];
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] = order_key(x[v]);
      top = max(top, key[v]);
    }
    top = group_max<L>(top);
    const bool open = top != 0;
    const float m = open ? key_value(top) : 0.f;

    // scores of all experts (over e^min(m, 0) or e^m), where something needs them; they
    // are not kept in registers during the choice
    bool routed = open;
    float z = 1.f;
    [[maybe_unused]] float f = 1.f;                // what makes them scores
    [[maybe_unused]] auto biased_keys = [&](const float (&s)[V]) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        key[v] = x[v] == -__builtin_inff() ? 0u : order_key(__builtin_fmaf(s[v], f, p.bias[min(e0 + v, p.E - 1)]));
    };
    if (BIASED || balance || (!p.renorm && !sigmoid)) {
      float s[V];
      z = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = shifted_score(x[v], m, sigmoid);
        z += s[v];
      }
      z = group_sum<L>(z);
      if (!open) z = 1.f;
      const float r = 1.f / z;
      if constexpr (BIASED) {
        f = sigmoid ? exp_nonpos(fminf(m, 0.f)) : r;
        biased_keys(s);
        bool some = false;                         // a bias of -inf may have closed the open ones
#pragma unroll
        for (int v = 0; v < V; ++v) some = some || key[v] != 0;
        routed = ((__ballot(some) >> base) & (L == 64 ? ~uint64_t(0) : uint64_t(0xFFFF))) != 0;
      }
      if (balance) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float pe = routed ? s[v] * r : 0.f;
          if constexpr (L == 16) {
            pe = across<16>(pe, [](float a, float b) { return a + b; });
            pe = across<32>(pe, [](float a, float b) { return a + b; });
          }
          if (lane < L) part[wave][v * L + l] += pe;
        }
      }
    }

    // lane j of the group takes choice j
    int id = -1;
    float xs = -__builtin_inff();
    auto take = [&](int j, uint32_t g, uint64_t who, int sel) {
      const int w = __builtin_ctzll(who >> base);       // the lowest lane of the group
      float xsel = 0.f;
      if constexpr (BIASED) xsel = __shfl(pick(x, sel), base + w, 64);
      else xsel = key_value(g);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (l == w && v == sel) key[v] = 0;
      sel = __shfl(sel, base + w, 64);
      if (l == j && g != 0) {
        id = w * V + sel;
        xs = xsel;
      }
    };
    // the largest key of the group, and where this lane has it first
    auto largest = [&](int& sel, uint64_t& who) {
      uint32_t best = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) best = max(best, key[v]);
      const uint32_t g = group_max<L>(best);
      who = __ballot(best == g);
      sel = 0;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) sel = key[v] == g ? v : sel;
      return g;
    };
    if constexpr (!BIASED) {
      for (int j = 0; j < p.k; ++j) {
        int sel;
        uint64_t who;
        const uint32_t g = largest(sel, who);
        take(j, g, who, sel);
      }
    } else {
      const float most = sigmoid ? 1.f : f;
      bool close = false;
      float before = 0.f;
      for (int j = 0; j <= p.k; ++j) {
        int sel;
        uint64_t who;
        const uint32_t g = largest(sel, who);
        const float now = key_value(g);
        if (j > 0 && g != 0) close = close || !(before - now > biased_tolerance(before, most, sigmoid));
        before = now;
        if (j < p.k) take(j, g, who, sel);
      }
      if (__ballot(close)) {
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = shifted_score(x[v], m, sigmoid);
        biased_keys(s);
        id = -1;
        double z64 = 1.0;
        if (!sigmoid) {
          z64 = 0.0;
#pragma unroll 1
          for (int v = 0; v < V; ++v) z64 += exp_nonpos(double(pick(x, v)) - double(m));
          z64 = group_sum<L>(z64);
        }
#pragma unroll 1
        for (int j = 0; j < p.k; ++j) {
          int sel;
          uint64_t who;
          const uint32_t g = largest(sel, who);
          const float now = key_value(g), cut = now - biased_tolerance(now, most, sigmoid);
          uint32_t near = 0;
#pragma unroll
          for (int v = 0; v < V; ++v) near |= uint32_t(key[v] != 0 && !(key_value(key[v]) < cut)) << v;
          if (__ballot(group_sum<L>(__popc(near)) > 1)) {
            uint64_t best = 0;
            while (__ballot(near != 0)) {
              const int v = near ? __builtin_ctz(near) : 0;
              const double xv = pick(x, v);
              const double e = exp_nonpos(sigmoid ? -__builtin_fabs(xv) : xv - double(m));
              const double sv = (sigmoid && xv > 0.0 ? 1.0 : e) / (sigmoid ? 1.0 + e : z64);
              const uint64_t kd = order_key(sv + double(p.bias[min(e0 + v, p.E - 1)]));
              if (near != 0 && kd > best) {
                best = kd;
                sel = v;
              }
              near &= near - 1;
            }
            who = __ballot(best == group_max<L>(best));
          }
          take(j, g, who, sel);
        }
      }
    }

    routed_sum += routed && l == 0;

    float w = 0.f;
    if (p.renorm) {
      uint32_t tc = l < p.k ? order_key(xs) : 0;
      tc = group_max<L>(tc);
      const float mc = tc ? key_value(tc) : 0.f;
      const float s = id >= 0 ? shifted_score(xs, mc, sigmoid) : 0.f;
      const float sum = group_sum<L>(s);
      w = id >= 0 ? p.scale * (s / sum) : 0.f;
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
  // over waves, in their order
  routed_sum = group_sum<64>(routed_sum);
  if (lane == 0) routed_of[wave] = routed_sum;
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) sum += part[w][e % V * L + e / V];
    p.part_sums[size_t(blockIdx.x) * p.E + e] = sum;
    p.part_counts[size_t(blockIdx.x) * p.E + e] = count[e];
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < kRouteWaves; ++w) n += routed_of[w];
    p.part_routed[blockIdx.x] = n;
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
  int sigmoid, renorm;
  float scale;
};

constexpr int kRouteBwdThreads = 256;

// dx = sum over choices of u_j at their experts, plus p times what the loss and, for
// softmax, the other scores take off:
//   shares q_j       u_j = scale q_j (dw_j - sum_i q_i dw_i) [(1 - s_j) for sigmoid]
//   softmax, plain   u_j = scale p_j dw_j, and - p_e sum_j u_j at every expert
//   sigmoid, plain   u_j = scale s_j (1 - s_j) dw_j
//   loss             f_e = dloss E / (k n^2) counts_e: p_e (f_e - sum p f) [(1 - s_e)]
// A token without choices, and rows of the logits that it alone would read, add
// nothing.  An expert that a token names twice gets both gradients.
template <bool BF16, int L, int V>
__device__ __forceinline__ void route_bwd_body(const RouteBwdArgs& p) {
  constexpr int PER_BLOCK = kRouteBwdThreads / L;
  const int lane = threadIdx.x & 63;
  const int l = lane & (L - 1), base = lane & ~(L - 1);
  const int e0 = l * V;
  const bool sigmoid = p.sigmoid != 0, whole = p.E % V == 0, loss = p.counts != nullptr;
  const long long t = (long long)block_index() * PER_BLOCK + threadIdx.x / L;
  const bool in = t < p.T;
  int id = in && l < p.k ? p.ids[t * p.k + l] : -1;
  if (id >= p.E) id = -1;
  const uint64_t any = __ballot(id >= 0) >> base;
  const bool routed = (L == 64 ? any : any & 0xFFFFu) != 0;
  float xs = -__builtin_inff(), dw = 0.f;
  if (id >= 0) {
    if constexpr (BF16) xs = __uint_as_float(uint32_t(static_cast<const uint16_t*>(p.x)[size_t(t) * p.E + id]) << 16);
    else xs = static_cast<const float*>(p.x)[size_t(t) * p.E + id];
    dw = p.scale * p.dw[t * p.k + l];
  }

  // what every expert gets: p_e (f_e - off)
  float pe[V], f[V], off = 0.f, z = 1.f, m = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) pe[v] = f[v] = 0.f;
  float x[V];
  const bool all = loss || !(p.renorm || sigmoid);
  if (all) {
    if (routed) {
      load_logits<BF16, V>(p.x, size_t(t) * p.E, e0, p.E, whole, x);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = -__builtin_inff();
    }
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) top = max(top, order_key(x[v]));
    top = group_max<L>(top);
    m = top ? key_value(top) : 0.f;
    z = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      pe[v] = shifted_score(x[v], m, sigmoid);
      z += pe[v];
    }
    z = group_sum<L>(z);
    if (top == 0) z = 1.f;                  // no expert of the row is open
    const float r = 1.f / z;
#pragma unroll
    for (int v = 0; v < V; ++v) pe[v] *= r;
    if (loss) {
      const double n = *p.routed;
      const float c = n > 0.0 ? float(double(*p.dloss) * p.E / (double(p.k) * n * n)) : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f[v] = c * float(p.counts[e0 + v < p.E ? e0 + v : 0]);
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
  if (id < 0) u = 0.f;

  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    d[v] = 0.f;
    if (all) {
      d[v] = pe[v] * (f[v] - off);
      if (sigmoid) d[v] *= one_minus_sigmoid(x[v]);
    }
  }
  for (int j = 0; j < p.k; ++j) {
    const int ej = __shfl(id, base + j, 64) - e0;
    const float uj = __shfl(u, base + j, 64);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (ej == v) d[v] += uj;
  }
  if (!in) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (e0 + v >= p.E) continue;
    const float o = routed ? d[v] : 0.f;
    if constexpr (BF16) static_cast<uint16_t*>(p.dx)[size_t(t) * p.E + e0 + v] = uint16_t(bf16_bits(o));
    else static_cast<float*>(p.dx)[size_t(t) * p.E + e0 + v] = o;
  }
}

}  // namespace dg
