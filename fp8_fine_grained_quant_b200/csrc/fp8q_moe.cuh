// fp8q_moe.cuh -- what surrounds the grouped GEMMs in a mixture-of-experts
// layer: the choice of experts from router logits and its gradient, the row
// layouts of the grouped GEMMs, the tokens quantized into them, and the
// weighted sum of the experts' outputs and its gradient.
//
// The pages name the two grouped layouts ("Deepgemm lancado no dia 4 da semana
// de codigo aberto Deepseek", "Principais caracteristicas") and the 1x128
// activation tiles ("The Insider Secrets Of Deepseek Discovered", Figure 7
// (a)); these kernels produce and consume those layouts.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "fp8q_codes.cuh"
#include "fp8q_ptx.cuh"
#include "fp8q_quant.cuh"

namespace fp8q {

constexpr int kMaxExperts = 1024;  // experts of a router or layout
constexpr int kMaxTopK = 32;       // experts of one token (one lane of a warp each)
constexpr int kMaxGroups = 32;     // expert groups (one lane each)

__device__ __forceinline__ double neg_inf_f64() { return __longlong_as_double(0xFFF0000000000000ll); }
__device__ __forceinline__ float neg_inf_f32() { return __int_as_float(0xFF800000); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

// ---------------------------------------------------------------------------
// Expert choice.  For each token with logits l over E experts:
//   score   p_e = softmax(l)_e or 1 / (1 + exp(-l_e));
//   key     p_e + bias_e with a bias, else p_e; where single experts are
//           compared without a bias, l_e itself (the same order);
//   groups  the E / n_group experts of a group share the group's best key or
//           the sum of its best two; the topk_group best groups stay;
//   choice  the top_k best keys of the experts that stay, best first;
//   weights scale * p_e, or scale * p_e / sum of the chosen p (renorm): the
//           bias moves the choice, not the weights.
// Equal keys (and groups) go to the lower index.  An expert whose logit or
// bias is -inf or NaN is never chosen; places that find no expert get id -1
// and weight 0.  A logit of +inf counts as the largest finite FP32.
//
// Two keys that differ by less than their FP32 error would make the choice
// depend on how the scores were evaluated, so keys are compared as binary64
// values; moe_route_kernel reaches the same choice in FP32 where it can prove it.
// ---------------------------------------------------------------------------
struct RouteArgs {
  const void* logits;  // [T, E] f32 or bf16
  const float* bias;   // [E] or null
  int32_t* ids;        // [T, top_k]
  float* weights;      // [T, top_k]
  int64_t T;
  int32_t E, top_k, n_group, topk_group, group_top;
  int32_t sigmoid, renorm;
  float scale;
};

// Logit e of a row as FP32; -inf for NaN, the largest finite value for +inf.
template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  float l;
  if constexpr (kBf16)
    l = __bfloat162float(static_cast<const __nv_bfloat16*>(row)[e]);
  else
    l = static_cast<const float*>(row)[e];
  if (!(l > neg_inf_f32())) return neg_inf_f32();
  return fminf(l, FLT_MAX);
}

template <bool kBf16>
__device__ __forceinline__ const void* logits_row(const void* logits, int64_t t, int E) {
  return static_cast<const uint8_t*>(logits) + t * E * (kBf16 ? 2 : 4);
}

// Weights of the chosen experts: lane j holds id (or -1) and returns its weight.
// Where a chosen sigmoid could underflow, its ratios are formed from
// e^(l - c) / (1 + e^l) with c = min(0, largest chosen logit), which stays
// finite and keeps the largest at 1/2 or more.  row_max and row_sum are the
// softmax statistics of the whole row (used without renorm).
__device__ __forceinline__ float route_weight(float l, bool found, bool sigmoid, bool renorm, float scale,
                                              float row_max, float row_sum) {
  float p;
  if (sigmoid) {
    p = div_full(1.0f, 1.0f + expf(-l));
    if (renorm && __any_sync(0xFFFFFFFFu, found && l < -64.0f)) {
      const float c = fminf(warp_max(found ? l : neg_inf_f32()), 0.0f);
      p = l > 0.0f ? p : div_full(expf(l - c), 1.0f + expf(l));
    }
  } else if (renorm) {
    p = expf(l - warp_max(found ? l : neg_inf_f32()));
  } else {
    p = div_full(expf(l - row_max), row_sum);
  }
  if (renorm) p = div_full(p, warp_sum(found ? p : 0.0f));
  return found ? scale * p : 0.0f;
}

// Scores in binary64.  Out of line: few rows need them, and one copy of the
// exponential keeps their code short (a cold path's time is its instruction
// fetches as much as its arithmetic).
__device__ __noinline__ double exp_f64(double x) { return exp(x); }
__device__ __noinline__ double score_f64(bool sigmoid, float l, float row_max, double sum) {
  const double x = exp_f64(sigmoid ? -static_cast<double>(l) : static_cast<double>(l) - static_cast<double>(row_max));
  return sigmoid ? 1.0 / (1.0 + x) : x / sum;
}

// The sum of exp(l - row_max) over a row in binary64.
template <bool kBf16>
__device__ __noinline__ double row_sum_f64(const void* row, int E, float row_max) {
  double sum = 0.0;
  for (int e = threadIdx.x & 31; e < E; e += 32) {
    const float l = load_logit<kBf16>(row, e);
    if (l > neg_inf_f32()) sum += exp_f64(static_cast<double>(l) - static_cast<double>(row_max));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
  return sum;
}

// The whole choice in binary64.  keys: the warp's E doubles of shared memory.
// Returns the id of place `lane` (or -1).
template <bool kBf16>
__device__ __noinline__ int route_choose_f64(const RouteArgs& a, const void* row, double* keys, float row_max) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  const int E = a.E;
  const double sum = a.sigmoid ? 0.0 : row_sum_f64<kBf16>(row, E, row_max);
  const bool by_score = a.bias != nullptr || (a.n_group > 1 && a.group_top == 2);
  for (int e = lane; e < E; e += 32) {
    const float l = load_logit<kBf16>(row, e);
    double k = static_cast<double>(l);
    if (by_score) {
      double p = score_f64(a.sigmoid, l, row_max, sum);
      if (a.bias != nullptr) p += static_cast<double>(__ldg(a.bias + e));
      k = l > neg_inf_f32() && p > neg_inf_f64() ? p : neg_inf_f64();
    }
    keys[e] = k + 0.0;  // -0 as +0
  }
  __syncwarp();
  if (a.n_group > 1) {
    const int size = E / a.n_group;
    int lanes = 32;  // of a group
    while (lanes * a.n_group > 32) lanes >>= 1;
    const int g = lane / lanes;
    double b1 = neg_inf_f64(), b2 = neg_inf_f64();
    if (g < a.n_group) {
#pragma unroll 4
      for (int i = lane & (lanes - 1); i < size; i += lanes) {
        const double k = keys[g * size + i];
        b2 = fmax(b2, fmin(b1, k));
        b1 = fmax(b1, k);
      }
    }
    for (int off = 1; off < lanes; off <<= 1) {
      const double o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, off), o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, off);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    const double total = a.group_top == 2 && b2 > neg_inf_f64() ? b1 + b2 : b1;
    int ahead = 0;
    for (int h = 0; h < a.n_group; ++h) {
      const double o = __shfl_sync(0xFFFFFFFFu, total, h * lanes);
      ahead += o > total || (o == total && h < g);
    }
    const uint32_t keep = __ballot_sync(0xFFFFFFFFu, g < a.n_group && ahead < a.topk_group);
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
      if (!((keep >> (e / size * lanes)) & 1u))
        keys[e] = neg_inf_f64();
      else if (by_score && a.bias == nullptr)
        keys[e] = static_cast<double>(load_logit<kBf16>(row, e)) + 0.0;
    }
    __syncwarp();
  }
  // the lane's best key and its expert (the first of equals)
  double best = neg_inf_f64();
  int at = E;
  auto rescan = [&] {
    best = neg_inf_f64();
    at = E;
    for (int e0 = lane; e0 < E; e0 += 32 * kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int e = e0 + 32 * i;
        const double k = e < E ? keys[e] : neg_inf_f64();
        if (k > best) {
          best = k;
          at = e;
        }
      }
    }
  };
  rescan();
  int mine = -1;
  for (int j = 0; j < a.top_k; ++j) {
    // order-preserving integers of the keys, the larger half first, then the lower expert
    const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(best));
    const unsigned long long o = bits ^ (bits >> 63 ? ~0ull : 0x8000000000000000ull);
    const uint32_t hi = static_cast<uint32_t>(o >> 32), lo = static_cast<uint32_t>(o);
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, at < E ? hi : 0u);
    if (top == 0u) break;  // no lane has a key
    bool in = at < E && hi == top;
    const uint32_t low = __reduce_max_sync(0xFFFFFFFFu, in ? lo : 0u);
    in = in && lo == low;
    const int w = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, in ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
    if (lane == j) mine = w;
    if (lane == (w & 31)) {  // the lane that scans w
      keys[w] = neg_inf_f64();
      rescan();
    }
    __syncwarp();
  }
  return mine;
}

// Largest and smallest value of a warp, one instruction each.
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float redux_min(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// N values in descending order, by an odd-even merge network (N a power of two).
template <int N>
__device__ __forceinline__ void sort_descending(float (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1) {
#pragma unroll
    for (int q = p; q >= 1; q >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i + q < N && i >= q % p && (i - q % p) / q % 2 == 0 && i / (2 * p) == (i + q) / (2 * p)) {
          const float x = v[i], y = v[i + q < N ? i + q : i];
          v[i] = fmaxf(x, y);
          v[i + q < N ? i + q : i] = fminf(x, y);
        }
      }
    }
  }
}

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// e^x for comparisons: 2^(x log2 e) by ex2.approx.ftz (2 ulp), the product
// rounded; off by at most (2 + |x|) 2^-23 relative.
__device__ __forceinline__ float exp_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
  return r;
}

// How the experts of a row lie over a warp: the lanes of group g are
// g << lanes_log2 and the next ones, each with `per_lane` consecutive experts
// of the group, so lane order is expert order.  With one group: 32 lanes.
struct RouteSplit {
  int32_t size;        // experts of a group
  int32_t lanes_log2;  // lanes of a group
  int32_t per_lane;    // at most the kernel's VPL
  int32_t vector;      // the lanes' runs tile the row and are aligned: vector loads
};

// A lane's logits as loaded: with vector loads VPL consecutive values, else
// one value a word (the type's -inf past the lane's share).
template <int VPL, bool kBf16>
__device__ __forceinline__ void load_share(const void* row, int base, int count, bool vector, uint32_t (&w)[VPL]) {
  constexpr int kSize = kBf16 ? 2 : 4;
  constexpr int kWords = VPL * kSize / 4;  // 0: too few for a word, never vector
  if (kWords > 0 && vector) {
    const uint8_t* p = static_cast<const uint8_t*>(row) + static_cast<int64_t>(base) * kSize;
    if constexpr (kWords >= 4) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
      }
    } else if constexpr (kWords == 2) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = x.x;
      w[1] = x.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if constexpr (kBf16)
        w[i] = i < count ? __ldg(static_cast<const uint16_t*>(row) + base + i) : 0xFF80u;
      else
        w[i] = i < count ? __ldg(static_cast<const uint32_t*>(row) + base + i) : 0xFF800000u;
    }
  }
}
template <int VPL, bool kBf16>
__device__ __forceinline__ void share_values(const uint32_t (&w)[VPL], bool vector, float (&l)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if constexpr (!kBf16)
      l[i] = __uint_as_float(w[i]);
    else if (VPL > 1 && vector)
      l[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
    else
      l[i] = __uint_as_float(w[i] << 16);
  }
}

// FP32 scores of the choice, and how far their keys may be off: key_reach is the
// least distance at which the keys a and b are surely in order.
template <bool kSigmoid>
__device__ __forceinline__ float score_f32(float l, float row_max, float inv_sum) {
  return kSigmoid ? rcp_approx(1.0f + exp_approx(-l)) : exp_approx(l - row_max) * inv_sum;
}
template <bool kSigmoid>
__device__ __forceinline__ float key_reach(float a, float b) {
  return (kSigmoid ? 0x1p-20f : 0x1p-17f) + 0x1p-22f * fmaxf(fabsf(a), fabsf(b));
}

// Whether every expert in [from, end) of the warp's lanes whose key lies in reach
// of expert `last`'s has its very logit and bias.  Out of line: few rows need it.
template <bool kBf16, bool kSigmoid>
__device__ __noinline__ bool border_is_equal(const void* row, const float* bias, int from, int end, int last,
                                             float row_max, float inv_sum) {
  const float ll = load_logit<kBf16>(row, last), lb = __ldg(bias + last);
  const float lk = score_f32<kSigmoid>(ll, row_max, inv_sum) + lb;
  bool equal = true;
  for (int e = from; e < end; ++e) {
    const float l = load_logit<kBf16>(row, e), b = __ldg(bias + e);
    if (!(l > neg_inf_f32() && b > neg_inf_f32())) continue;  // never chosen
    const float k = score_f32<kSigmoid>(l, row_max, inv_sum) + b;
    equal = equal && ((l == ll && b == lb) || fabsf(k - lk) > key_reach<kSigmoid>(k, lk));
  }
  return __all_sync(0xFFFFFFFFu, equal);
}

constexpr int kExactVpl = 8;  // up to this share, a comparison that FP32 leaves open is settled in registers
constexpr int kRouteWarps = 4;
constexpr int kRouteCtasPerSm = 8;  // up to eight experts a lane: 64 registers

// The common case in FP32, with a proof: a warp holds its row in registers,
// each lane its share's keys in descending order.  A round of the choice takes
// the largest of the lanes' heads (one warp reduction); the lowest lane that
// has it gives it up.  A warp walks rows at a stride of the grid, the next
// row's logits loaded while it chooses from the current one.
//
// Without a bias experts are compared by their logits, exactly.  With one, and
// for group sums, FP32 keys are compared, and each comparison that decides
// (neighbours in the choice, the first expert left out, the worst group kept
// against the best one dropped) must be wider than the keys' error.  Equal keys
// of equal logits and biases need no proof among the chosen; where the first one
// left out equals the last chosen, every key in reach must (border_is_equal).
// Where one is not (about one row in a thousand), the keys within reach of the
// comparison are evaluated in binary64, a key a lane: the best of every group, or
// the chosen and those next to the last of them.  Shares above eight experts, and
// more than 32 keys in reach, take route_choose_f64.
//
// Bound by instruction issue (about 810 a row of 256 experts, half of them on the
// integer and compare pipe), not by its bytes: 32768 rows of 256 experts in 8
// groups, biased sigmoid, take 37.0 us on a B200 against 5.5 us for reading them;
// 4096 rows of 32 take 3.1 us and one row 3.1 us, a launch's time.  Rows of nothing
// but equal keys, which border_is_equal reads again, take 46 us for 32768 of 256
// without groups, 117 where the groups are equal too.  (All keys in
// binary64: 121 us; a row that left its choice to route_choose_f64 alone held up
// the launch's end by 7 us.)  The errors, by exp_approx's:
//   sigmoid  p (1 - p) (2 + |x|) 2^-23 <= 2^-23, + 2^-24 from 1 + e and 2^-23
//            from rcp: below 2^-21.6 a key; + 2^-24 |key| from adding the bias;
//   softmax  at most 30 * 2^-23 of p from the row's sum (37 additions, and
//            sum p |x| <= ln 1024), and 3 * 2^-23: below 2^-17.9 for any two
//            keys, as their p sum to at most 1;
// so two keys further apart than 2^-20 (sigmoid) or 2^-17 (softmax) + 2^-22 of
// the larger are in order, and a sum of two keys is off by at most that tolerance
// and 2^-20 of its larger key (2^-22 from both keys, 2^-23 from the sum and from
// adding the bound to it).
template <int VPL, bool kBf16, bool kSigmoid, bool biased>
__global__ void __launch_bounds__(32 * kRouteWarps, VPL <= 8 ? kRouteCtasPerSm : 1)
    moe_route_kernel(RouteArgs a, RouteSplit sp) {
  extern __shared__ double route_keys[];  // [kRouteWarps][E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> sp.lanes_log2;
  const int first = (lane & ((1 << sp.lanes_log2) - 1)) * sp.per_lane;
  const int base = g * sp.size + first;
  const int count = g < a.n_group ? max(0, min(sp.per_lane, sp.size - first)) : 0;
  const bool pair_sums = a.n_group > 1 && a.group_top == 2;
  const bool stats = !kSigmoid && (biased || pair_sums || !a.renorm);  // something needs the row's softmax
  constexpr float tol = kSigmoid ? 0x1p-20f : 0x1p-17f;
  float bias[biased ? VPL : 1];  // -inf: never chosen
  if constexpr (biased) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      bias[i] = i < count ? __ldg(a.bias + base + i) : 0.0f;
      if (!(bias[i] > neg_inf_f32())) bias[i] = neg_inf_f32();
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  uint32_t raw[VPL];
  if (t < a.T) load_share<VPL, kBf16>(logits_row<kBf16>(a.logits, t, a.E), base, count, sp.vector, raw);
  for (; t < a.T; t += step) {
    const void* row = logits_row<kBf16>(a.logits, t, a.E);
    float l[VPL];
    share_values<VPL, kBf16>(raw, sp.vector, l);
    if (t + step < a.T)
      load_share<VPL, kBf16>(logits_row<kBf16>(a.logits, t + step, a.E), base, count, sp.vector, raw);
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = fminf(fmaxf(l[i], neg_inf_f32()), FLT_MAX);  // NaN to -inf
    float row_max = neg_inf_f32(), row_sum = 0.0f;
    if (stats) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) row_max = fmaxf(row_max, l[i]);
      row_max = redux_max(row_max);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (l[i] > neg_inf_f32()) row_sum += a.renorm ? exp_approx(l[i] - row_max) : expf(l[i] - row_max);
      }
      row_sum = warp_sum(row_sum);
    }
    const float inv_sum = rcp_approx(row_sum);
    auto score = [&](float x) { return score_f32<kSigmoid>(x, row_max, inv_sum); };

    // keys: the logits (-0 as +0), or score + bias; -inf: never chosen
    float key[VPL], s[VPL];
    if constexpr (!biased) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = l[i] + 0.0f;
    } else {
      float least = l[0];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        key[i] = score(l[i]) + bias[i];
        least = fminf(least, l[i]);
      }
      if (least == neg_inf_f32()) {  // the sigmoid of -inf is 0, of a masked row's softmax NaN
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = l[i] == neg_inf_f32() ? neg_inf_f32() : key[i];
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = key[i];
    sort_descending<VPL>(s);

    bool certain = true;
    bool stays = true;  // the lane's group is kept
    if (a.n_group > 1) {
      // the group's best one or two, in every lane of the group
      float b1 = s[0], b2 = VPL > 1 ? s[VPL > 1 ? 1 : 0] : neg_inf_f32();
      for (int off = 1; off < (1 << sp.lanes_log2); off <<= 1) {
        const float o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, off), o2 = __shfl_xor_sync(0xFFFFFFFFu, b2, off);
        b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
        b1 = fmaxf(b1, o1);
      }
      float total = b1;  // group_top 1: the best key decides
      float mag = fabsf(b1);  // the largest magnitude in it (of a sum of scores, which do not cancel, below 1)
      if (pair_sums) {
        const float v1 = biased ? b1 : score(b1), v2 = biased ? b2 : score(b2);
        total = b1 == neg_inf_f32() ? b1 : (b2 == neg_inf_f32() ? v1 : v1 + v2);
        mag = biased ? (b2 == neg_inf_f32() ? mag : fmaxf(mag, -b2)) : 1.0f;
      }
      // groups ahead of this one, a share of the comparisons in each of its lanes
      const int lanes = 1 << sp.lanes_log2;
      int ahead = 0;
      for (int h0 = 0; h0 < a.n_group; h0 += lanes) {
        const int h = h0 + (lane & (lanes - 1));
        const float o = __shfl_sync(0xFFFFFFFFu, total, h << sp.lanes_log2);
        ahead += h < a.n_group && (o > total || (o == total && h < g));
      }
      for (int off = 1; off < lanes; off <<= 1) ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, off);
      const bool in = g < a.n_group;
      bool keep = in && ahead < a.topk_group;
      if ((pair_sums || biased) && a.topk_group < a.n_group) {
        // each total's least and largest possible value: it is off by as much as its keys are, and they may cancel
        const float err = tol + 0x1p-20f * mag;
        const float w = redux_min(keep ? fmaxf(total - err, neg_inf_f32()) : __int_as_float(0x7F800000));
        // (-inf only for a group without a key: a sum below FP32's range is one of the least finite ones)
        const float least = b1 > neg_inf_f32() ? -FLT_MAX : neg_inf_f32();
        const float b = redux_max(in && !keep ? fmaxf(total + err, least) : neg_inf_f32());
        if (!(b == neg_inf_f32() || w > b)) {
          if constexpr (VPL <= kExactVpl) {
            // the groups' sums in binary64, of the keys that can be among their best: each lane's
            // next largest in turn while some lane has one
            const double sum = kSigmoid ? 0.0 : row_sum_f64<kBf16>(row, a.E, row_max);
            const float last = a.group_top == 2 ? b2 : b1;
            const bool margin = biased && fabsf(last) <= FLT_MAX;  // logits compare exactly
            const float from = margin ? last - 2.0f * (tol + 0x1p-22f * fabsf(last)) : last;
            double d1 = neg_inf_f64(), d2 = neg_inf_f64();
            uint32_t used = 0u;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
              const bool can = s[j] > neg_inf_f32() && s[j] >= from;
              if (!__any_sync(0xFFFFFFFFu, can)) break;
              int at = -1;  // the lane's first unused key s[j]
#pragma unroll
              for (int i = 0; i < VPL; ++i)
                if (at < 0 && key[i] == s[j] && !((used >> i) & 1u)) at = i;
              if (can) {
                used |= 1u << at;
                double v = score_f64(kSigmoid, load_logit<kBf16>(row, base + at), row_max, sum);
                if constexpr (biased) v += static_cast<double>(__ldg(a.bias + base + at));
                d2 = fmax(d2, fmin(d1, v));
                d1 = fmax(d1, v);
              }
            }
            for (int off = 1; off < lanes; off <<= 1) {
              const double o1 = __shfl_xor_sync(0xFFFFFFFFu, d1, off), o2 = __shfl_xor_sync(0xFFFFFFFFu, d2, off);
              d2 = fmax(fmin(d1, o1), fmax(d2, o2));
              d1 = fmax(d1, o1);
            }
            const double sum2 = a.group_top == 2 && d2 > neg_inf_f64() ? d1 + d2 : d1;
            ahead = 0;
            for (int h = 0; h < a.n_group; ++h) {
              const double o = __shfl_sync(0xFFFFFFFFu, sum2, h << sp.lanes_log2);
              ahead += o > sum2 || (o == sum2 && h < g);
            }
            keep = in && ahead < a.topk_group;
          } else {
            certain = false;
          }
        }
      }
      stays = keep;
      if (!keep) s[0] = neg_inf_f32();  // the lane never gives up a key
    }

    // the choice: lane j gets place j's key and the lane that had it; with a
    // bias also the first expert left out
    float my_key = neg_inf_f32();
    int my_lane = 0;
    auto place = [&](int j, float m) {
      const int w = __ffs(__ballot_sync(0xFFFFFFFFu, s[0] == m)) - 1;
      if (lane == j) {
        my_key = m;
        my_lane = w;
      }
      const bool mine = lane == w;
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = mine ? (i + 1 < VPL ? s[i + 1 < VPL ? i + 1 : i] : neg_inf_f32()) : s[i];
    };
    const int rounds = a.top_k + (biased && a.top_k < 32 ? 1 : 0);
    for (int j = 0; j < rounds; ++j) {
      const float m = redux_max(s[0]);
      if (m == neg_inf_f32()) break;
      place(j, m);
    }
    int id = -1;
    float lid = 0.0f;  // its logit
    auto find = [&] {
      const bool placed = my_key > neg_inf_f32();
      // equal keys of one lane come one after another, in expert order: how many went before this one
      const float prev = __shfl_up_sync(0xFFFFFFFFu, my_key, 1);
      const int prev_lane = __shfl_up_sync(0xFFFFFFFFu, my_lane, 1);
      const uint32_t repeats =
          __ballot_sync(0xFFFFFFFFu, lane > 0 && placed && my_key == prev && my_lane == prev_lane);
      int seen = 0;
      if (repeats != 0u) seen = lane - (31 - __clz(~repeats & (0xFFFFFFFFu >> (31 - lane))));
      int at = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const bool hit = __shfl_sync(0xFFFFFFFFu, key[i], my_lane) == my_key;
        if (hit && seen == 0) at = i;
        seen -= hit;
      }
      if (placed) {
        id = (my_lane >> sp.lanes_log2) * sp.size + (my_lane & ((1 << sp.lanes_log2) - 1)) * sp.per_lane + at;
        lid = load_logit<kBf16>(row, id);
      }
    };
    find();
    if constexpr (biased) {
      float next = __shfl_down_sync(0xFFFFFFFFu, my_key, 1);
      const float rest = a.top_k == 32 ? redux_max(s[0]) : neg_inf_f32();  // of 32 places, the first expert left out
      if (lane == 31) next = rest;
      bool sure = true;
      if (lane < a.top_k && next > neg_inf_f32())
        sure = my_key - next > key_reach<kSigmoid>(my_key, next);
      if (certain && !__all_sync(0xFFFFFFFFu, sure)) {
        // keys in one another's reach: certain only between equal logits with equal biases
        float bid = id >= 0 ? __ldg(a.bias + id) : 0.0f;
        const float nl = __shfl_down_sync(0xFFFFFFFFu, lid, 1), nb = __shfl_down_sync(0xFFFFFFFFu, bid, 1);
        certain = __all_sync(0xFFFFFFFFu, sure || (lane < 31 && lid == nl && bid == nb));
        if (certain && !((__ballot_sync(0xFFFFFFFFu, sure) >> (a.top_k - 1)) & 1u)) {
          // the first expert left out equals the last chosen, so it stands for none of those behind it
          const int end = stays ? base + count : base;
          certain = border_is_equal<kBf16, kSigmoid>(row, a.bias, base, end, __shfl_sync(0xFFFFFFFFu, id, a.top_k - 1),
                                                     row_max, inv_sum);
        }
        if (VPL <= kExactVpl && !certain && a.top_k < 32) {
          // more places, until the next key cannot reach the last that counts
          const float kth = __shfl_sync(0xFFFFFFFFu, my_key, a.top_k - 1);
          const float reach = kth - 2.0f * (tol + 0x1p-22f * fabsf(kth));
          float m = redux_max(s[0]);
          for (int j = rounds; j < 32 && m > neg_inf_f32() && m >= reach; ++j) {
            place(j, m);
            m = redux_max(s[0]);
          }
          if (!(m > neg_inf_f32() && m >= reach)) {  // all within reach have a lane
            find();
            bid = id >= 0 ? __ldg(a.bias + id) : 0.0f;
            // their keys in binary64, one a lane, and their order
            const double sum = kSigmoid ? 0.0 : row_sum_f64<kBf16>(row, a.E, row_max);
            const double v =
                id >= 0 ? score_f64(kSigmoid, lid, row_max, sum) + static_cast<double>(bid) : neg_inf_f64();
            const int n = __popc(__ballot_sync(0xFFFFFFFFu, id >= 0));
            int ahead = 0, mine = -1;
            for (int j = 0; j < n; ++j) {
              const double o = __shfl_sync(0xFFFFFFFFu, v, j);
              const int oi = __shfl_sync(0xFFFFFFFFu, id, j);
              ahead += o > v || (o == v && oi < id);
            }
            for (int j = 0; j < n; ++j) {
              const int oa = __shfl_sync(0xFFFFFFFFu, ahead, j), oi = __shfl_sync(0xFFFFFFFFu, id, j);
              if (oa == lane) mine = oi;
            }
            id = mine;
            lid = id >= 0 ? load_logit<kBf16>(row, id) : 0.0f;
            certain = true;
          }
        }
      }
    }
    if (!certain) {
      id = route_choose_f64<kBf16>(a, row, route_keys + static_cast<int64_t>(warp) * a.E, row_max);
      lid = id >= 0 ? load_logit<kBf16>(row, id) : 0.0f;
      __syncwarp();
    }
    const bool found = id >= 0 && lane < a.top_k;
    const float w = route_weight(lid, found, kSigmoid, a.renorm, a.scale, row_max, row_sum);
    if (lane < a.top_k) {
      a.ids[t * a.top_k + lane] = id;
      a.weights[t * a.top_k + lane] = w;
    }
  }
}

// Every row in binary64: for splits that leave a lane more experts than the
// register kernel holds.
template <bool kBf16>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_f64_kernel(RouteArgs a) {
  extern __shared__ double route_keys[];  // [kRouteWarps][E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= a.T) return;
  const void* row = logits_row<kBf16>(a.logits, t, a.E);
  float row_max = neg_inf_f32(), row_sum = 0.0f;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += 32) row_max = fmaxf(row_max, load_logit<kBf16>(row, e));
    row_max = warp_max(row_max);
    for (int e = lane; e < a.E; e += 32) {
      const float l = load_logit<kBf16>(row, e);
      if (l > neg_inf_f32()) row_sum += expf(l - row_max);
    }
    row_sum = warp_sum(row_sum);
  }
  const int id = route_choose_f64<kBf16>(a, row, route_keys + static_cast<int64_t>(warp) * a.E, row_max);
  const float l = id >= 0 ? load_logit<kBf16>(row, id) : 0.0f;
  const float w = route_weight(l, id >= 0, a.sigmoid, a.renorm, a.scale, row_max, row_sum);
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = w;
  }
}

// ---------------------------------------------------------------------------
// Gradient of the weights with respect to the logits (the choice itself is
// constant).  With g the gradient of the weights, over the chosen j:
//   softmax, renorm:  r = softmax over the chosen;  dl_j = scale r_j (g_j - <g, r>)
//   sigmoid, renorm:  r = p / sum p;                dl_j = scale r_j (g_j - <g, r>) (1 - p_j)
//   sigmoid:          dl_j = scale g_j p_j (1 - p_j)
//   softmax:          dl_e = scale p_e (d_e - <g, p>), d_e = the g of e, 0 where e was not chosen
// Every other logit gets 0.  Places with an id outside [0, E) count for
// nothing; an id that appears twice gets the sum.  1 - p_j is evaluated as
// 1 / (1 + exp(l_j)), which keeps its digits when p_j is close to 1.
//
// One warp per token.  The chosen experts' values are scattered into a row of
// shared memory and read back in expert order; only the dense form reads the
// whole row of logits, once, into registers.  Bound by the latency of one row a
// warp: 16384 rows of 160 take 8.4 us on a B200 in the dense form, 3.3 us for
// their bytes.
// ---------------------------------------------------------------------------
struct RouteBwdArgs {
  const void* logits;
  const int32_t* ids;
  const float* dweights;
  void* dlogits;
  int64_t T;
  int32_t E, top_k, sigmoid, renorm;
  float scale;
};

// VPL: experts of a lane (lane, lane + 32, ...), E <= 32 VPL; kDense: softmax
// without renorm, where every logit gets a gradient.
template <int VPL, bool kBf16, bool kDense>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_bwd_kernel(RouteBwdArgs a) {
  extern __shared__ float route_grad[];  // [kRouteWarps][E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= a.T) return;
  float* d = route_grad + static_cast<int64_t>(warp) * E;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (i * 32 + lane < E) d[i * 32 + lane] = 0.0f;
  const void* row = logits_row<kBf16>(a.logits, t, E);
  float x[kDense ? VPL : 1];
  if constexpr (kDense) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = i * 32 + lane < E ? load_logit<kBf16>(row, i * 32 + lane) : neg_inf_f32();
  }
  int id = lane < a.top_k ? __ldg(a.ids + t * a.top_k + lane) : -1;
  if (id >= E) id = -1;
  float g = 0.0f, l = neg_inf_f32();
  if (id >= 0) {
    g = __ldg(a.dweights + t * a.top_k + lane);
    if constexpr (!kDense) l = load_logit<kBf16>(row, id);
  }
  // dense: p is 0 where the logit is -inf, so its gradient counts for nothing
  const bool has = id >= 0 && (kDense || l > neg_inf_f32());
  float v = g;  // dense: the gradient of p; else of the logit
  if constexpr (!kDense) {
    const float not_p = a.sigmoid ? 1.0f / (1.0f + expf(l)) : 1.0f;
    if (a.renorm) {
      const float r = route_weight(l, has, a.sigmoid, true, 1.0f, 0.0f, 1.0f);
      const float mean = warp_sum(has ? g * r : 0.0f);
      v = a.scale * r * (g - mean) * not_p;
    } else {
      v = a.scale * g * (1.0f / (1.0f + expf(-l))) * not_p;
    }
  }
  if (!has) v = 0.0f;
  // an id that appears more than once: the sum, in place order
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, has ? id : -1 - lane);
  if (__any_sync(0xFFFFFFFFu, __popc(same) > 1)) {
    float total = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
      const float o = __shfl_sync(0xFFFFFFFFu, v, j);
      if ((same >> j) & 1u) total += o;
    }
    v = total;
  }
  __syncwarp();  // the row is zero
  if (has) d[id] = v;
  __syncwarp();
  float o[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) o[i] = i * 32 + lane < E ? d[i * 32 + lane] : 0.0f;
  if constexpr (kDense) {
    float m = neg_inf_f32();
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, x[i]);
    m = redux_max(m);
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] = x[i] > neg_inf_f32() ? expf(x[i] - m) : 0.0f;
      o[i] = x[i] > 0.0f ? o[i] : 0.0f;  // not 0 times a gradient of inf or NaN
      sum += x[i];
      dot = fmaf(x[i], o[i], dot);
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const float mean = dot * inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = a.scale * (x[i] * inv) * (o[i] - mean);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    if (e < E) {
      if constexpr (kBf16)
        static_cast<__nv_bfloat16*>(a.dlogits)[t * E + e] = __float2bfloat16_rn(o[i]);
      else
        static_cast<float*>(a.dlogits)[t * E + e] = o[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Row layouts of the grouped GEMMs from the chosen experts.  Entry i = t *
// top_k + j of ids goes to the row
//   contiguous:  128 * (whole blocks of the experts before) + rank,
//   masked:      expert * cap + rank (no row, -1, once the rank reaches cap),
// rank being the number of earlier entries with the same expert, so the layout
// does not depend on any order of execution.  Ids outside [0, E) get no row.
//
// One cluster of up to eight CTAs (1024 threads each) takes all entries; every
// warp owns one run of consecutive entries.  It counts its run's experts into
// its own row of a shared table (the lanes of 32 entries with equal ids find
// one another by a vote per bit of the id, so no two lanes touch one counter),
// the table's columns are turned into exclusive prefixes over the warps, the
// CTAs' totals are read from one another's shared memory, and the warps hand out
// ranks, from registers where a run is short.  One launch and no atomics.  For
// many entries a launch before it counts the experts of each chunk into a
// workspace, and the CTAs of this one, no cluster, sum those.  On a B200: 4.9 us
// for 488 entries, 8.0 for 32768 (latency: barriers and a few hundred dependent
// steps), 11 to 13 for 262144, 104 for 8388608.
// ---------------------------------------------------------------------------
struct LayoutArgs {
  const int32_t* ids;
  int64_t n;          // entries
  int32_t E;
  int64_t cap;        // masked: rows of an expert; 0: contiguous
  int32_t* slots;     // [n]
  int32_t* m_indices; // contiguous: [blocks]
  int64_t blocks;
  int32_t* counts;    // contiguous: entries of each expert; masked: min(entries, cap)
  int32_t* chunk_counts;  // [CTAs][E]: the first launch's counts; null: one cluster
};

// Above this many entries eight SMs are too few for them: the layout takes two
// launches, a CTA per kLayoutChunk entries or, from one CTA an SM on, per equal
// share of them (every CTA sums all CTAs' counts, so more CTAs cost their
// square: 8388608 entries of 256 experts take 104 us in 148 shares, 1000 in
// chunks of 4096), and a workspace.  (32768 entries: 8.1 us in one cluster, 8.9 in two
// launches; 262144: 58 against 13.5, when both were measured.)
constexpr int64_t kLayoutClusterMax = 32768;
constexpr int kLayoutChunk = 4096;
constexpr int kLayoutMaxChunks = 148;
constexpr int64_t layout_chunks(int64_t n) {
  const int64_t c = (n + kLayoutChunk - 1) / kLayoutChunk;
  return c < kLayoutMaxChunks ? c : kLayoutMaxChunks;
}

constexpr int kLayoutThreads = 1024;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kLayoutMaxCtas = 8;  // the portable cluster size
constexpr int kLayoutAhead = 4;    // groups of 32 entries loaded together
constexpr int layout_smem(int E) { return kLayoutWarps * E * 4; }

// Groups of 32 entries that each warp of `ctas` CTAs takes.
__host__ __device__ constexpr int64_t layout_groups(int64_t n, int64_t ctas) {
  return (n + kLayoutThreads * ctas - 1) / (kLayoutThreads * ctas);
}

// The lanes that hold the same id; `bits` covers every id and -1.
__device__ __forceinline__ uint32_t same_lanes(int e, int bits) {
  uint32_t same = 0xFFFFFFFFu;
  for (int b = 0; b < bits; ++b) {
    const bool set = (e >> b) & 1;
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, set);
    same &= set ? v : ~v;
  }
  return same;
}

// First launch of a large layout: the entries of each expert in each chunk of
// `chunk` entries (integer shared-memory atomics: their order does not change a
// count).
__global__ void __launch_bounds__(kLayoutThreads) moe_layout_count_kernel(const int32_t* __restrict__ ids, int64_t n,
                                                                          int64_t chunk, int32_t E,
                                                                          int32_t* __restrict__ counts) {
  __shared__ int32_t hist[kMaxExperts];
  const int tid = threadIdx.x;
  hist[tid] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * chunk, to = from + chunk < n ? from + chunk : n;
  for (int64_t i0 = from + tid; i0 < to; i0 += kLayoutChunk) {
    int e[kLayoutChunk / kLayoutThreads];
#pragma unroll
    for (int k = 0; k < kLayoutChunk / kLayoutThreads; ++k) {
      const int64_t i = i0 + k * kLayoutThreads;
      e[k] = i < to ? __ldg(ids + i) : -1;
    }
#pragma unroll
    for (int k = 0; k < kLayoutChunk / kLayoutThreads; ++k)
      if (static_cast<uint32_t>(e[k]) < static_cast<uint32_t>(E)) atomicAdd(&hist[e[k]], 1);
  }
  __syncthreads();
  if (tid < E) counts[static_cast<int64_t>(blockIdx.x) * E + tid] = hist[tid];
}

__global__ void __launch_bounds__(kLayoutThreads) moe_layout_kernel(LayoutArgs a) {
  extern __shared__ int32_t layout_table[];  // [kLayoutWarps][E]
  __shared__ int32_t hist[kMaxExperts];      // this CTA's entries of each expert
  __shared__ int32_t before[kMaxExperts];    // entries in the CTAs ahead
  __shared__ int32_t start[kMaxExperts + 1]; // contiguous: first block of each expert
  __shared__ int32_t warp_total[kLayoutWarps];
  const auto cluster = cooperative_groups::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.E, bits = 33 - __clz(E - 1);  // of the ids below E, and one that only -1 has
  int32_t* mine = layout_table + warp * E;
  // groups of 32 entries of a warp, its first entry, and the CTA's warps that have any
  const int64_t groups = layout_groups(a.n, gridDim.x);
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kLayoutWarps + warp) * groups * 32 + lane;
  const int64_t left = a.n - static_cast<int64_t>(blockIdx.x) * kLayoutWarps * groups * 32;
  const int warps = left <= 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(kLayoutWarps),
                                                         (left + groups * 32 - 1) / (groups * 32)));
  auto expert = [&](int64_t g) {
    const int64_t i = first + g * 32;
    const int e = g < groups && i < a.n ? __ldg(a.ids + i) : -1;
    return static_cast<uint32_t>(e) < static_cast<uint32_t>(E) ? e : -1;
  };
  int e[kLayoutAhead];
  uint32_t same[kLayoutAhead];
#pragma unroll
  for (int k = 0; k < kLayoutAhead; ++k) e[k] = expert(k);
  for (int i = tid; i < warps * E; i += kLayoutThreads) layout_table[i] = 0;
  __syncthreads();
  if (warp < warps) {
    for (int64_t g = 0; g < groups; g += kLayoutAhead) {
      if (g > 0) {
#pragma unroll
        for (int k = 0; k < kLayoutAhead; ++k) e[k] = expert(g + k);
      }
#pragma unroll
      for (int k = 0; k < kLayoutAhead; ++k) same[k] = g + k < groups ? same_lanes(e[k], bits) : 0u;
#pragma unroll
      for (int k = 0; k < kLayoutAhead; ++k) {
        if (e[k] >= 0 && lane == __ffs(same[k]) - 1) mine[e[k]] += __popc(same[k]);
        __syncwarp();
      }
    }
  }
  __syncthreads();
  int32_t count = 0, ahead = 0;
  if (tid < E) {
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int32_t c = layout_table[w * E + tid];
      layout_table[w * E + tid] = count;
      count += c;
    }
    hist[tid] = count;
  }
  if (a.chunk_counts != nullptr) {
    if (tid < E) {
      count = 0;
#pragma unroll 8
      for (unsigned r = 0; r < gridDim.x; ++r) {
        const int32_t h = __ldg(a.chunk_counts + static_cast<int64_t>(r) * E + tid);
        if (r < blockIdx.x) ahead += h;
        count += h;
      }
    }
  } else if (gridDim.x > 1) {
    cluster.sync();
    if (tid < E) {
      int32_t h[kLayoutMaxCtas];
#pragma unroll
      for (unsigned r = 0; r < kLayoutMaxCtas; ++r)
        h[r] = r < gridDim.x ? *cluster.map_shared_rank(&hist[tid], r) : 0;
      count = 0;
#pragma unroll
      for (unsigned r = 0; r < kLayoutMaxCtas; ++r) {
        if (r < blockIdx.x) ahead += h[r];
        count += h[r];
      }
    }
    cluster.sync();  // no CTA may end while another reads its counts
  }
  if (tid < E) before[tid] = ahead;
  // exclusive prefix of the experts' blocks of 128 rows
  const int size = (count + 127) >> 7;
  int incl = size;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int own = warp_total[lane];
    int s = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, s, off);
      if (lane >= off) s += o;
    }
    warp_total[lane] = s - own;
  }
  __syncthreads();
  start[tid] = warp_total[warp] + incl - size;
  if (tid == kLayoutThreads - 1) start[kMaxExperts] = warp_total[warp] + incl;
  if (blockIdx.x == 0 && tid < E)
    a.counts[tid] = a.cap > 0 && count > a.cap ? static_cast<int32_t>(a.cap) : count;
  __syncthreads();
  if (warp < warps) {
    for (int64_t g = 0; g < groups; g += kLayoutAhead) {
      if (groups > kLayoutAhead) {  // else still in registers
#pragma unroll
        for (int k = 0; k < kLayoutAhead; ++k) e[k] = expert(g + k);
#pragma unroll
        for (int k = 0; k < kLayoutAhead; ++k) same[k] = g + k < groups ? same_lanes(e[k], bits) : 0u;
      }
#pragma unroll
      for (int k = 0; k < kLayoutAhead; ++k) {
        int64_t slot = -1;
        if (e[k] >= 0) {
          const int64_t r = static_cast<int64_t>(before[e[k]]) + mine[e[k]] + __popc(same[k] & ((1u << lane) - 1u));
          if (a.cap > 0)
            slot = r < a.cap ? e[k] * a.cap + r : -1;
          else
            slot = static_cast<int64_t>(start[e[k]]) * 128 + r;
        }
        __syncwarp();
        if (e[k] >= 0 && lane == __ffs(same[k]) - 1) mine[e[k]] += __popc(same[k]);
        __syncwarp();
        if (g + k < groups && first + (g + k) * 32 < a.n) a.slots[first + (g + k) * 32] = static_cast<int32_t>(slot);
      }
    }
  }
  if (a.cap == 0) {
    // the expert of each block: the last whose first block is not past it
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kLayoutThreads;
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * kLayoutThreads + tid; b < a.blocks; b += stride) {
      int owner = -1;
      if (b < start[kMaxExperts]) {
        int lo = 0, hi = kMaxExperts;  // start[lo] <= b < start[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (start[mid] <= b) lo = mid; else hi = mid;
        }
        owner = lo;
      }
      a.m_indices[b] = owner;
    }
  }
}

// ---------------------------------------------------------------------------
// Rows of the contiguous layout that no entry fills: in the last block of each
// expert, the rows past its count.  Where the next block has another expert, the
// block is its expert's last.  The last block of the buffer may end before its
// expert's run does (fewer rows than the layout needs: the slots beyond are
// skipped), so there the block's place in the run, which starts at the first block
// with an index of e or more, says which entries it holds.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool is_pad_row(int64_t row, const int32_t* m_indices, const int32_t* counts, int E,
                                           int64_t blocks) {
  const int64_t b = row >> 7;
  const int e = m_indices[b];
  if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(E)) return false;
  if (b + 1 < blocks) {
    if (m_indices[b + 1] == e) return false;
    const int rest = counts[e] & 127;
    return rest != 0 && static_cast<int>(row & 127) >= rest;
  }
  int64_t lo = 0, hi = b;  // the run's first block lies in [lo, hi]
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (m_indices[mid] < e) lo = mid + 1; else hi = mid;
  }
  return (b - lo) * 128 + (row & 127) >= counts[e];
}

// ---------------------------------------------------------------------------
// Dispatch: the 1x128 quantization of each token's tiles (the same codes and
// scales as quant_act_1x128_kernel, bit for bit), each tile written to the
// rows of the token's slots.  A token is quantized once however many experts
// it goes to.  Slots outside [0, rows) are skipped; pad rows of the contiguous
// layout (m_indices given) get codes 0 and scales 1; other rows stay as they
// are.  Eight lanes own a tile, as in the quantizer.  HBM-bound: 4096 tokens of
// 7168 channels to 8 of 32 experts take 57.7 us on a B200 (335 MB with the pad
// rows, 5.8 TB/s), 61 tokens 2.8 us.
// ---------------------------------------------------------------------------
struct DispatchArgs {
  const uint8_t* x;    // [T, D] bf16
  const int32_t* slots;
  int32_t top_k;
  int32_t nkb;         // D / 128
  int64_t num_tiles;   // T * nkb
  int64_t rows;
  const int32_t* m_indices;  // or null
  const int32_t* counts;
  int32_t E;
  uint8_t* q;          // [rows, D]
  float* s;            // [rows, nkb]
};

__global__ void __launch_bounds__(256, 5) moe_dispatch_1x128_kernel(DispatchArgs a) {
  const int sub = threadIdx.x & 7;
  const int64_t D = static_cast<int64_t>(a.nkb) * 128;
  const int64_t grp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const int64_t ngrp = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 3;
  // same trip count for every lane of a warp (the shuffles need all 32)
  for (int64_t t = grp; (t & ~int64_t(3)) < a.num_tiles; t += ngrp) {
    const bool valid = t < a.num_tiles;
    uint32_t v[8];
    if (valid)
      ld_nc_v8(a.x + t * 256 + sub * 32, v);
    else
      zero8(v);
    float amax = abs_max16(v);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
    const float sc = group_scale(amax);
    if (valid) {
      const uint4 codes = codes16_bf16(v, sc);
      const uint32_t tok = static_cast<uint32_t>(t) / static_cast<uint32_t>(a.nkb);
      const uint32_t kb = static_cast<uint32_t>(t) - tok * static_cast<uint32_t>(a.nkb);
      const int32_t* sl = a.slots + static_cast<int64_t>(tok) * a.top_k;
      for (int j = 0; j < a.top_k; ++j) {
        const int64_t row = __ldg(sl + j);
        if (row >= 0 && row < a.rows) {
          *reinterpret_cast<uint4*>(a.q + row * D + static_cast<int64_t>(kb) * 128 + sub * 16) = codes;
          if (sub == 0) a.s[row * a.nkb + kb] = sc;
        }
      }
    }
  }
  if (a.m_indices != nullptr) {
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    for (int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; row < a.rows;
         row += nwarps) {
      if (!is_pad_row(row, a.m_indices, a.counts, a.E, a.rows >> 7)) continue;
      for (int64_t c = lane; c < D / 16; c += 32)
        *reinterpret_cast<uint4*>(a.q + row * D + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      for (int c = lane; c < a.nkb; c += 32) a.s[row * a.nkb + c] = 1.0f;
    }
  }
}

// ---------------------------------------------------------------------------
// Combine: out[t] = sum over j of w[t, j] * y[slot[t, j]] in FP32, rounded
// once to bf16.  Without weights the plain sum: the gradient of the dispatch
// with respect to its tokens.  Entries without a row count for nothing; a
// token with none gets zeros.  A thread owns eight channels of a token and
// loads them from four rows at once (61 tokens of 7168 channels, top-8: 2.8 us on
// a B200; row by row 3.6).
// ---------------------------------------------------------------------------
struct CombineArgs {
  const uint8_t* y;      // [rows, D] bf16
  const int32_t* slots;  // [T, top_k]
  const float* weights;  // [T, top_k] or null
  uint8_t* out;          // [T, D] bf16
  int32_t top_k;
  int32_t nkb;
  int64_t num_tiles;     // T * nkb
  int64_t rows;
};

// acc[0..7] += w * the eight bf16 of v.
__device__ __forceinline__ void fma8_bf16(float (&acc)[8], const uint4& v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xFFFF0000u), acc[2 * i + 1]);
  }
}

constexpr int kCombineEntries = 4;  // rows of a token loaded together

__global__ void __launch_bounds__(256) moe_combine_kernel(CombineArgs a) {
  const int sub = threadIdx.x & 15;  // eight channels of a 128-channel tile
  const int64_t stride = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 4;
  const int64_t D = static_cast<int64_t>(a.nkb) * 128;
  for (int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4; t < a.num_tiles; t += stride) {
    const uint32_t tok = static_cast<uint32_t>(t) / static_cast<uint32_t>(a.nkb);
    const uint32_t kb = static_cast<uint32_t>(t) - tok * static_cast<uint32_t>(a.nkb);
    const int64_t e0 = static_cast<int64_t>(tok) * a.top_k;
    const int64_t col = static_cast<int64_t>(kb) * 128 + sub * 8;
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < a.top_k; j0 += kCombineEntries) {
      uint4 v[kCombineEntries];
      float w[kCombineEntries];
#pragma unroll
      for (int j = 0; j < kCombineEntries; ++j) {
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        w[j] = 0.0f;
        if (j0 + j < a.top_k) {
          const int64_t row = __ldg(a.slots + e0 + j0 + j);
          if (row >= 0 && row < a.rows) {
            v[j] = ld_nc_v4(a.y + (row * D + col) * 2);
            w[j] = a.weights != nullptr ? __ldg(a.weights + e0 + j0 + j) : 1.0f;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kCombineEntries; ++j) fma8_bf16(acc, v[j], w[j]);
    }
    *reinterpret_cast<uint4*>(a.out + t * 256 + sub * 16) =
        make_uint4(bf16x2_rn(acc[0], acc[1]), bf16x2_rn(acc[2], acc[3]), bf16x2_rn(acc[4], acc[5]),
                   bf16x2_rn(acc[6], acc[7]));
  }
}

// ---------------------------------------------------------------------------
// Gradient of the combine: dy[slot[t, j]] = bf16(w[t, j] * dout[t]) and
// dw[t, j] = <dout[t], y[slot[t, j]]> (FP32 sums; 0 where the entry has no
// row).  Pad rows of the contiguous layout (m_indices given) get zeros, other
// rows stay as they are.  One CTA per token: a thread holds eight channels of
// dout and walks the token's rows, eight entries at a time with their partial
// dot products in registers, which are then summed over the CTA in a fixed
// order.  HBM-bound: 4096 tokens of 7168 channels, top-8, take 165 us on a B200
// (998 MB and 33 MB of pad rows, 6.3 TB/s); with each row's load used before the
// next was issued they took 217.
// ---------------------------------------------------------------------------
struct CombineBwdArgs {
  const uint8_t* dout;   // [T, D] bf16
  const uint8_t* y;      // [rows, D] bf16
  const int32_t* slots;
  const float* weights;
  uint8_t* dy;           // [rows, D] bf16
  float* dweights;       // [T, top_k]
  int32_t top_k;
  int64_t T, D, rows;
  const int32_t* m_indices;  // or null
  const int32_t* counts;
  int32_t E;
};

__device__ __forceinline__ float dot8_bf16(float acc, const uint4& x, const uint4& y) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), acc);
    acc = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), acc);
  }
  return acc;
}

// The eight bf16 of v times w, each rounded once.
__device__ __forceinline__ uint4 scale8_bf16(const uint4& v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = bf16x2_rn(__fmul_rn(w, __uint_as_float(u[i] << 16)), __fmul_rn(w, __uint_as_float(u[i] & 0xFFFF0000u)));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int kCombineBwdThreads = 256;
constexpr int kCombineBwdEntries = 8;  // entries of a token handled at once

__global__ void __launch_bounds__(kCombineBwdThreads, 3) moe_combine_bwd_kernel(CombineBwdArgs a) {
  constexpr int kWarps = kCombineBwdThreads / 32;
  __shared__ float part[kWarps][kCombineBwdEntries];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t chunks = a.D / 8;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const uint8_t* dout = a.dout + t * a.D * 2;
    for (int j0 = 0; j0 < a.top_k; j0 += kCombineBwdEntries) {
      int32_t row[kCombineBwdEntries];
      float w[kCombineBwdEntries], acc[kCombineBwdEntries];
#pragma unroll
      for (int j = 0; j < kCombineBwdEntries; ++j) {
        row[j] = -1;
        w[j] = acc[j] = 0.0f;
        if (j0 + j < a.top_k) {
          const int32_t r = __ldg(a.slots + t * a.top_k + j0 + j);
          if (r >= 0 && r < a.rows) row[j] = r;
          w[j] = __ldg(a.weights + t * a.top_k + j0 + j);
        }
      }
      for (int64_t c = tid; c < chunks; c += kCombineBwdThreads) {
        const uint4 g = ld_nc_v4(dout + c * 16);
        uint4 v[kCombineBwdEntries];  // all rows' loads before any is used
#pragma unroll
        for (int j = 0; j < kCombineBwdEntries; ++j) {
          v[j] = make_uint4(0u, 0u, 0u, 0u);
          if (row[j] >= 0) v[j] = ld_nc_v4(a.y + (row[j] * a.D + c * 8) * 2);
        }
#pragma unroll
        for (int j = 0; j < kCombineBwdEntries; ++j) {
          if (row[j] < 0) continue;
          acc[j] = dot8_bf16(acc[j], g, v[j]);
          *reinterpret_cast<uint4*>(a.dy + (row[j] * a.D + c * 8) * 2) = scale8_bf16(g, w[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kCombineBwdEntries; ++j) {
        const float s = warp_sum(acc[j]);
        if (lane == 0) part[warp][j] = s;
      }
      __syncthreads();
      if (tid < kCombineBwdEntries && j0 + tid < a.top_k) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += part[i][tid];
        a.dweights[t * a.top_k + j0 + tid] = s;
      }
      __syncthreads();
    }
  }
  if (a.m_indices != nullptr) {
    const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp; row < a.rows; row += nwarps) {
      if (!is_pad_row(row, a.m_indices, a.counts, a.E, a.rows >> 7)) continue;
      for (int64_t c = lane; c < chunks; c += 32)
        *reinterpret_cast<uint4*>(a.dy + (row * a.D + c * 8) * 2) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

}  // namespace fp8q
