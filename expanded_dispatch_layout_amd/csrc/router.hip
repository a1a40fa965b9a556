// moe_router, moe_router_backward: the choice of each token's experts from the
// gate's logits, and its gradient.
//
//   s = softmax(x) or 1 / (1 + exp(-x));  the topk largest s + bias, the lowest
//   expert first among equals;  w_k = s_k, or s_k / sum of the chosen s
//
// -inf and NaN logits are experts that are not available: score 0, never
// chosen.  +inf counts as the largest finite value.
//
// The choice.  Without a bias and groups the logits are compared, and no exponential is
// needed to choose.  Otherwise the keys s + bias, and the
// groups' sums of two, are compared in fp64: fp32 scores are off by a few
// 2^-24, and neighbouring keys of 256 experts are nearer than that in one row
// out of some thousands, which would then go to another expert.
//
// The weights.  Normalised weights are formed without the common factor that
// can underflow: exp(x - max) over the chosen for softmax, and for the sigmoid,
// which is exp(min(x, 0)) / (1 + exp(-|x|)), the same with min(x, 0).
//
// Keys in fp32 first, exact ones where those leave a choice open: choose_quickly,
// choose_closely and choose_exactly, the last without any limit on groups or ties
// (16384 rows of 160 experts in 8 groups, which are not 2^n lanes: 93 us).
//
// Memory is not what bounds it: 16384 rows of 256 experts with bias and groups, 8
// chosen, are 18 MB, 4 us at a copy's rate, and take 18.6 us; the 256 keys and the
// choices are 373 vector instructions a row.  Its gradient, 34 MB: 12.8 us.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "common.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kMaxGroups = 64;

__device__ __forceinline__ float load_logit(const void* x, bool f32, int64_t at) {
  const float v = f32 ? ((const float*)x)[at] : bf16_to_f32(((const uint16_t*)x)[at]);
  return v != v ? -INFINITY : fminf(v, FLT_MAX);
}
__device__ __forceinline__ float load_bias(const float* __restrict__ bias, int e) {
  if (!bias) return 0.f;
  const float b = bias[e];
  return b != b ? -INFINITY : fminf(b, FLT_MAX);
}
__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
// The largest key of the wave and its expert, the lowest among equals; -1 where
// every key is -inf.
template <typename T>
__device__ __forceinline__ void wave_best(T& key, int& at) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const T k = __shfl_xor(key, o, kWave);
    const int a = __shfl_xor(at, o, kWave);
    if (k > key || (k == key && a < at)) {
      key = k;
      at = a;
    }
  }
}

// The value that one lane holds (the same number of a lane for all).
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}

struct Sizes {
  int E, topk, groups, topk_groups;
  bool f32, sigmoid, normalize;
};

typedef float v4f __attribute__((ext_vector_type(4)));

// kPer fp32 logits or biases, 16 bytes at a time; NaN becomes -inf.
template <int kPer>
__device__ __forceinline__ void load_wide(const float* p, float (&x)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; i += 4) {
    const v4f v = *reinterpret_cast<const v4f*>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i + j] = fminf(fmaxf(v[j], -INFINITY), FLT_MAX);
  }
}

// Logits of experts kPer lane + 0 .. kPer - 1; -inf past the last.
template <int kPer>
__device__ __forceinline__ void load_row(const void* __restrict__ logits, const Sizes& z,
                                         int64_t row_at, int lane, float (&x)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * lane + i;
    x[i] = e < z.E ? load_logit(logits, z.f32, row_at + e) : -INFINITY;
  }
}

// Logits that are compared as they are: -0 becomes +0, which it is equal to.
template <int kPer>
__device__ __forceinline__ void one_zero(float (&x)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] += 0.0f;
}

// Scores' common factor of a row: maximum and sum of softmax.
template <int kPer>
__device__ __forceinline__ void softmax_stats(const float (&x)[kPer], float& top, float& total) {
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = fmaxf(top, x[i]);
  top = wave_max_f(top);
  total = 0.f;
  if (top == -INFINITY) return;
#pragma unroll
  for (int i = 0; i < kPer; ++i) total += expf(x[i] - top);
  total = wave_sum_f(total);
}

// Weight of the expert this lane holds the id of (logit v, id < 0: none).
__device__ __forceinline__ float weight_of(float v, int id, const Sizes& z, float top,
                                           float total) {
  const bool here = id >= 0;
  if (!z.normalize) {
    if (!here) return 0.f;
    return z.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - top) / total;
  }
  const float low = here ? (z.sigmoid ? fminf(v, 0.f) : v) : -INFINITY;
  const float m = wave_max_f(low);
  float w = here ? expf(low - m) : 0.f;
  if (z.sigmoid && here) w /= 1.0f + expf(-fabsf(v));
  const float sum = wave_sum_f(w);
  return here ? w / sum : 0.f;
}

template <typename T, int kPer>
__device__ __forceinline__ int choose(T (&key)[kPer], const Sizes& z, int lane) {
  int mine = -1;
  for (int k = 0; k < z.topk; ++k) {
    T best = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 64 * i;
      }
    wave_best(best, at);
    if (best == (T)-INFINITY) break;
    if (lane == k) mine = at;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 64 * i == at) key[i] = -INFINITY;
  }
  return mine;
}

// The choice of one row by exact keys: the logits themselves, or fp64 scores.
template <int kPer>
__device__ __forceinline__ int choose_exactly(const void* __restrict__ logits, int64_t row_at,
                                              const float* __restrict__ bias, const Sizes& z,
                                              int lane) {
  float x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < z.E ? load_logit(logits, z.f32, row_at + e) : -INFINITY;
  }
  if (!bias && z.groups == 1) return choose<float, kPer>(x, z, lane);
  double key[kPer];
  double top = 0.0, sum = 1.0;
  if (!z.sigmoid) {
    float t = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) t = fmaxf(t, x[i]);
    t = wave_max_f(t);
    if (t == -INFINITY) return -1;
    top = t;
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += exp((double)x[i] - top);
    sum = wave_sum_d(sum);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    key[i] = -INFINITY;
    if (x[i] == -INFINITY) continue;
    key[i] = z.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i])) : exp((double)x[i] - top) / sum;
    if (bias) {
      const float b = bias[lane + 64 * i];
      key[i] = b != b ? -INFINITY : key[i] + (double)fminf(b, FLT_MAX);
    }
  }
  if (z.groups > 1) {
    const int per = z.E / z.groups;
    double group = -INFINITY;  // lane g: the sum of group g's two largest keys
    for (int g = 0; g < z.groups; ++g) {
      double first = -INFINITY, second = -INFINITY;
      int at = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + 64 * i;
        if (e / per != g || !(key[i] > -INFINITY)) continue;
        if (key[i] > first) {
          second = first;
          first = key[i];
          at = e;
        } else if (key[i] > second) {
          second = key[i];
        }
      }
      double best = first;
      int best_at = at;
      wave_best(best, best_at);
      if (best == -INFINITY) continue;
      double rest = best_at == at ? second : first;
      int none = 0;
      wave_best(rest, none);
      if (lane == g) group = rest > -INFINITY ? best + rest : best;
    }
    uint64_t chosen = 0;
    for (int k = 0; k < z.topk_groups; ++k) {
      double best = group;
      int at = group > -INFINITY ? lane : 0x7fffffff;
      wave_best(best, at);
      if (best == -INFINITY) break;
      chosen |= 1ull << at;
      if (lane == at) group = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (!(chosen >> ((lane + 64 * i) / per & 63) & 1)) key[i] = -INFINITY;
  }
  return choose<double, kPer>(key, z, lane);
}

// How far an fp32 key s + b may be from its exact value, in units of 2^-24 for
// s <= 1.  exp's argument is off by two half steps, which cost at most 2 * x e^-x /
// (1 + e^-x)^2 < 0.5 for the sigmoid and 2 * x e^-x < 0.8 for softmax; exp itself 2,
// of which the sigmoid takes a quarter; 1 + e 1; the reciprocal and product 3;
// softmax's sum of up to 16 values in a lane and 6 rounds of lanes 22.  So below 5 and
// 29; 8 and 64 are taken.  The sum with b: 1 of the key; 4 is taken.
__device__ __forceinline__ float key_error(float key, bool sigmoid) {
  return (sigmoid ? 0x1p-21f : 0x1p-18f) + 0x1p-22f * fabsf(key);
}
// fp32 key of one expert; top and inv: softmax's maximum and one over its sum.
__device__ __forceinline__ float quick_key(float v, float b, const Sizes& z, float top,
                                           float inv) {
  return (z.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-v)) : __expf(v - top) * inv) + b;
}
// Does an expert of logit v and bias b come before one of v2 and b2 that was lined up
// behind it, for certain?  The same logit and bias make the same key, and were lined up by
// their numbers.
__device__ __forceinline__ bool before(float v, float b, float v2, float b2, bool keys,
                                       const Sizes& z, float top, float inv) {
  if (v == v2 && b == b2) return true;
  if (!keys) return v > v2;
  const float k = quick_key(v, b, z, top, inv), k2 = quick_key(v2, b2, z, top, inv);
  return k - k2 > key_error(k, z.sigmoid) + key_error(k2, z.sigmoid);
}
// fp32 as unsigned numbers of the same order; no finite number is 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)~((int)u >> 31) | 0x80000000u));
}

// How far a group's sum of its two largest keys may be off: by both keys' errors (of
// which a sum that cancels shows nothing) and its own rounding, 1; 4 is taken.  The
// errors grow more slowly than the keys, so that this holds also where other two are the
// largest exactly.
__device__ __forceinline__ float sum_error(float first, float second, float sum, bool sigmoid) {
  return key_error(first, sigmoid) + (second > -INFINITY ? key_error(second, sigmoid) : 0.f) +
         0x1p-22f * fabsf(sum);
}
// Groups of 2^n lanes (kPer experts to a lane): each lane's two largest keys, then
// its group's.  Returns the sum of the group's two, -inf without any; rank: how
// many groups come before it; error (fp32 keys): sum_error.
// In fp32 a sum past the range stays finite: biases of the lowest value are still keys.
__device__ __forceinline__ float sum_of_two(float a, float b) {
  return fminf(fmaxf(a + b, -FLT_MAX), FLT_MAX);
}
__device__ __forceinline__ double sum_of_two(double a, double b) { return a + b; }
template <typename T, int kPer>
__device__ __forceinline__ T rank_groups(const T (&key)[kPer], const Sizes& z, int lane,
                                         int lanes, int& rank, float& error) {
  T m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    m2 = max(m2, min(m1, key[i]));
    m1 = max(m1, key[i]);
  }
  for (int o = 1; o < lanes; o <<= 1) {
    const T o1 = __shfl_xor(m1, o, kWave), o2 = __shfl_xor(m2, o, kWave);
    m2 = max(min(m1, o1), max(m2, o2));
    m1 = max(m1, o1);
  }
  const T sum = m2 > (T)-INFINITY ? sum_of_two(m1, m2) : m1;
  if constexpr (std::is_same<T, float>::value) error = sum_error(m1, m2, sum, z.sigmoid);
  rank = 0;
  for (int g = 0; g < z.groups; ++g) {
    const T other = lane_value(sum, g * lanes);
    rank += other > sum || (other == sum && g < lane / lanes);
  }
  return sum;
}

// Can the key of a smaller number, exactly, be the larger one's or more?  (By what the
// two numbers' lost bits leave open: the smallest distance of the two.)
template <uint32_t kIndex>
__device__ __forceinline__ bool may_pass(uint32_t small, uint32_t large, bool keys,
                                         const Sizes& z) {
  const float hi = unordered(large & ~kIndex), lo = unordered(small | kIndex);
  return hi - lo <= (keys ? key_error(hi, z.sigmoid) + key_error(lo, z.sigmoid) : 0.f);
}

// Without a bias but with groups the fp64 scores are in the order of the logits, unless
// fp64 holds two of them as one number: near 1 (sigmoid), below its range, or next to each
// other.  Is that possible for the logit of `mine` and that of `next`, or, where these are
// the same, another one below it?  (Scores that are told apart here differ by 2^-34 of
// themselves, of 1 for the sigmoid: 2^18 steps of fp64.)
template <uint32_t kIndex>
__device__ __forceinline__ bool one_score(uint32_t mine, uint32_t next, const Sizes& z,
                                          float top) {
  const uint32_t at = mine & ~kIndex;
  const float hi = unordered(at);
  const float lo = at != (next & ~kIndex) ? unordered(next | kIndex)
                                          : unordered(at - (z.f32 ? 1u : 0x10000u));
  const float slope = z.sigmoid ? __expf(-fmaxf(hi, 0.f)) : 1.f;
  return !((hi - lo) * slope > 0x1p-32f && lo - (z.sigmoid ? 0.f : top) > -600.f);
}

// The choice by fp32 keys.  A key is an ordered number whose low bits are
// replaced by the expert, counted down, so that a maximum of 32-bit numbers finds
// both, and equal ones by the lowest expert.  Lane l holds experts kPer l + 0 ..
// kPer - 1.  Sets `unsure` where two neighbours of the order, down to the first one
// left out, may lie nearer than the keys' errors (cut bits included) and turn out so by
// their whole keys, but for equal logits with equal biases: the row is then chosen
// exactly.  Of those left out, all that may reach the last one chosen are looked at.
template <int kPer>
__device__ __forceinline__ int choose_quickly(const float (&x)[kPer],
                                              const void* __restrict__ logits, int64_t row_at,
                                              const float* __restrict__ bias, const Sizes& z,
                                              int lane, bool& unsure) {
  constexpr uint32_t kIndex = 64 * kPer - 1;  // bits of an expert
  const bool scores = bias || z.groups > 1;
  float key[kPer];
  float top = 0.f, inv = 1.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = x[i];
  if (scores) {
    if (!z.sigmoid) {
      float t = x[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) t = fmaxf(t, x[i]);
      top = wave_max_f(t);
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) total += __expf(x[i] - top);
      inv = __builtin_amdgcn_rcpf(wave_sum_f(total));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (x[i] == -INFINITY) continue;
      key[i] = quick_key(x[i], load_bias(bias, kPer * lane + i), z, top, inv);
    }
  }
  unsure = false;
  if (z.groups > 1) {
    const int lanes = z.E / z.groups / kPer;
    int rank;
    float error;
    const float sum = rank_groups<float, kPer>(key, z, lane, lanes, rank, error);
    // The least that a group chosen may have, and the most of one left out.
    if (z.topk_groups < z.groups) {
      const bool group = lane < z.groups * lanes && sum > -INFINITY;
      const float least = -wave_max_f(group && rank < z.topk_groups ? error - sum : -INFINITY);
      const float most = wave_max_f(group && rank >= z.topk_groups ? sum + error : -INFINITY);
      unsure = most > -INFINITY && !(least > most);
    }
    if (rank >= z.topk_groups) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) key[i] = -INFINITY;
    }
  }
  // Without a bias the order is the logits', also between the groups chosen, if no two
  // have one score.
  const bool by_logits = !bias && z.groups > 1;
  if (by_logits) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = key[i] > -INFINITY ? x[i] : -INFINITY;
  }
  uint32_t u[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    u[i] = key[i] > -INFINITY
               ? (ordered(key[i]) & ~kIndex) | (kIndex - (uint32_t)(kPer * lane + i))
               : 0u;
  uint32_t mine = 0, next = 0;  // lane k: the k-th and the one after it
  for (int k = 0; k <= z.topk; ++k) {
    uint32_t best = u[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = max(best, u[i]);
    best = wave_max_u(best);
    if (lane == k) mine = best;
    if (lane == k - 1) next = best;
    if (best == 0) break;
#pragma unroll
    for (int i = 0; i < kPer; ++i) u[i] = u[i] == best ? 0u : u[i];
  }
  const bool here = lane < z.topk && mine != 0;
  const int id = here ? (int)(kIndex - (mine & kIndex)) : -1;
  if (here && next != 0 && may_pass<kIndex>(next, mine, bias != nullptr, z)) {
    const int other = (int)(kIndex - (next & kIndex));
    unsure |= !before(load_logit(logits, z.f32, row_at + id), load_bias(bias, id),
                      load_logit(logits, z.f32, row_at + other), load_bias(bias, other),
                      bias != nullptr, z, top, inv);
  }
  if (by_logits && here && next != 0) unsure |= one_score<kIndex>(mine, next, z, top);
  const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)mine, z.topk - 1);
  const uint32_t out = (uint32_t)__builtin_amdgcn_readlane((int)next, z.topk - 1);
  if (out != 0 && may_pass<kIndex>(out, last, bias != nullptr, z)) {
    const int at = (int)(kIndex - (last & kIndex));
    const float v = load_logit(logits, z.f32, row_at + at), b = load_bias(bias, at);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (u[i] != 0 && may_pass<kIndex>(u[i], last, bias != nullptr, z))
        unsure |= !before(v, b, x[i], load_bias(bias, kPer * lane + i), bias != nullptr, z, top,
                          inv);
  }
  unsure = __ballot(unsure) != 0;
  return id;
}

// The same by fp64 keys, for rows that fp32 leaves open.  Rounding the keys to the
// ordered numbers keeps their order but for equal ones: all that reach the topk-th
// are lined up, one to a lane, and ranked by the keys themselves.  Returns false
// where they are more than the lanes (many equal keys).
template <int kPer>
__device__ __forceinline__ bool choose_closely(const float (&x)[kPer],
                                               const float* __restrict__ bias, const Sizes& z,
                                               int lane, int& id) {
  constexpr uint32_t kIndex = 64 * kPer - 1;
  const bool scores = bias || z.groups > 1;
  double key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = x[i];
  if (scores) {
    double top = 0.0, total = 1.0;
    if (!z.sigmoid) {
      float t = x[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) t = fmaxf(t, x[i]);
      top = wave_max_f(t);
      total = 0.0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (x[i] > -INFINITY) total += exp((double)x[i] - top);
      total = wave_sum_d(total);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (x[i] == -INFINITY) continue;
      key[i] = z.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i])) : exp((double)x[i] - top) / total;
      if (bias) {
        const float b = bias[kPer * lane + i];
        key[i] = b != b ? -INFINITY : key[i] + (double)fminf(b, FLT_MAX);
      }
    }
  }
  if (z.groups > 1) {
    int rank;
    float unused;
    rank_groups<double, kPer>(key, z, lane, z.E / z.groups / kPer, rank, unused);
    if (rank >= z.topk_groups) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) key[i] = -INFINITY;
    }
  }
  uint32_t u[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    u[i] = key[i] > -INFINITY ? (ordered((float)key[i]) & ~kIndex) |
                                    (kIndex - (uint32_t)(kPer * lane + i))
                              : 0u;
  double mine = -INFINITY;  // lane c: the c-th candidate
  int expert = -1;
  uint32_t least = 0;  // what the topk-th one's number is
  int count = 0;
  for (;; ++count) {
    uint32_t best = u[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = max(best, u[i]);
    best = wave_max_u(best);
    if (best == 0 || (count >= z.topk && (best & ~kIndex) < least)) break;
    if (count == kWave) return false;
    if (count == z.topk - 1) least = best & ~kIndex;
    double own = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (u[i] == best) {
        own = key[i];
        u[i] = 0;
      }
    const int e = (int)(kIndex - (best & kIndex));
    own = lane_value(own, e / kPer);
    if (lane == count) {
      mine = own;
      expert = e;
    }
  }
  int rank = 0;
  for (int c = 0; c < count; ++c) {
    const double other = lane_value(mine, c);
    rank += other > mine || (other == mine && __builtin_amdgcn_readlane(expert, c) < expert);
  }
  id = -1;
  for (int c = 0; c < count; ++c)
    if (__builtin_amdgcn_readlane(rank, c) == lane) id = __builtin_amdgcn_readlane(expert, c);
  if (lane >= z.topk) id = -1;
  return true;
}

// One row by a whole wave.  kQuick: fp32 keys have been or are to be tried.
template <int kPer, bool kQuick>
__device__ __forceinline__ void route_row(const void* __restrict__ logits, int64_t stride,
                                          const float* __restrict__ bias, const Sizes& z,
                                          int64_t r, int lane, bool tried,
                                          int32_t* __restrict__ ids,
                                          float* __restrict__ weights) {
  float x[kPer];
  load_row<kPer>(logits, z, r * stride, lane, x);
  if (!bias) one_zero(x);
  int id = -1;
  bool unsure = true;
  if constexpr (kQuick) {
    if (!tried) id = choose_quickly<kPer>(x, logits, r * stride, bias, z, lane, unsure);
    if (unsure) unsure = !choose_closely<kPer>(x, bias, z, lane, id);
  }
  if (unsure) id = choose_exactly<kPer>(logits, r * stride, bias, z, lane);
  float top = 0.f, total = 1.f;
  if (!z.sigmoid && !z.normalize) softmax_stats<kPer>(x, top, total);
  float v = 0.f;
  if (id >= 0) v = load_logit(logits, z.f32, r * stride + id);
  const float w = weight_of(v, id, z, top, total);
  if (lane < z.topk) {
    ids[r * z.topk + lane] = id;
    weights[r * z.topk + lane] = w;
  }
}

template <int kPer, bool kQuick>
__global__ __launch_bounds__(kThreads) void router_kernel(
    const void* __restrict__ logits, int64_t stride, const float* __restrict__ bias, Sizes z,
    const int32_t* __restrict__ psum_rank, int nsrc, int64_t rows, int32_t* __restrict__ ids,
    float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nv = valid_rows(psum_rank, nsrc, rows);
  for (int64_t r = (int64_t)blockIdx.x * kWaves + wid; r < nv;
       r += (int64_t)gridDim.x * kWaves)
    route_row<kPer, kQuick>(logits, stride, bias, z, r, lane, false, ids, weights);
}

// Reductions of 16 lanes, by rotations: the result is in every lane.
template <typename F>
__device__ __forceinline__ int row_reduce(int v, F&& f) {
  v = f(v, dpp_move<0x128, 0xf>(v, v));  // row_ror:8
  v = f(v, dpp_move<0x124, 0xf>(v, v));
  v = f(v, dpp_move<0x122, 0xf>(v, v));
  v = f(v, dpp_move<0x121, 0xf>(v, v));
  return v;
}
__device__ __forceinline__ uint32_t row_max_u(uint32_t v) {
  return (uint32_t)row_reduce((int)v,
                              [](int a, int b) { return (int)max((uint32_t)a, (uint32_t)b); });
}
__device__ __forceinline__ float row_max_f(float v) {
  return __int_as_float(row_reduce(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}
__device__ __forceinline__ float row_sum_f(float v) {
  return __int_as_float(row_reduce(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

// The k-th largest number, given the one before it and the largest distance from
// it (wrapped round): 0 once there is none.
__device__ __forceinline__ uint32_t below(int k, uint32_t before, uint32_t distance) {
  return k > 0 && before == 0 ? 0u : before + distance;
}

// Key of one expert in fp64; softmax, which is only compared with its own row
// here, without its sum.
__device__ __forceinline__ double exact_key(float v, float b, const Sizes& z, float top) {
  return z.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) + (double)b : exp((double)v - (double)top);
}

// Four rows to a wave, 16 lanes each, for up to 14 choices out of up to 256
// experts: the reductions of a choice are half as long and serve four rows
// (16384 rows of 256 experts, 8 chosen: 24.5 us, 33 with a wave to a row).  The
// choice is choose_quickly's, with kPer experts to a lane.  What it leaves open is
// settled by fp64 keys of the few that matter; where these do not do, a row is
// taken by the whole wave afterwards (with rows left to that whenever two keys are
// near, 24.5 us in place of 20 for one in 170: whoever has one ends last; one in 70 may
// have near ones).
// The next choice is found without taking the last one out: of all numbers minus
// the last maximum, wrapped round, the largest is the next one below it.
// (Numbers of 0, which no expert has, are below all: there are some wherever the
// experts do not suffice.)
template <int kPer>
__global__ __launch_bounds__(kThreads) void router_quad_kernel(
    const void* __restrict__ logits, int64_t stride, const float* __restrict__ bias, Sizes z,
    bool wide_loads, const int32_t* __restrict__ psum_rank, int nsrc, int64_t rows,
    int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr uint32_t kIndex = 16 * kPer - 1;
  const int lane = threadIdx.x & 63, ql = lane & 15;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nv = valid_rows(psum_rank, nsrc, rows);
  const bool scores = bias || z.groups > 1;
  // Are numbers other than their keys?  (bf16 logits keep all their bits.)
  const bool loose = bias || z.f32;
  // Can a lane tell an exact key by itself?  (Softmax's sum would be fp64, too.)
  const bool exact = z.sigmoid || !bias;
  float b[kPer];
  if (bias && wide_loads) {
    load_wide<kPer>(bias + kPer * ql, b);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = kPer * ql + i;
      b[i] = bias && e < z.E ? bias[e] : 0.f;
      b[i] = fminf(fmaxf(b[i], -INFINITY), FLT_MAX);  // NaN: -inf
    }
  }
  for (int64_t r0 = ((int64_t)blockIdx.x * kWaves + wid) * 4; r0 < nv;
       r0 += (int64_t)gridDim.x * kWaves * 4) {
    const int64_t r = min(r0 + (lane >> 4), nv - 1);  // rows past the last: the last again
    const bool real = r0 + (lane >> 4) < nv;
    const int64_t at = r * stride + kPer * ql;
    float x[kPer];
    if (wide_loads) {  // fp32, every expert there
      load_wide<kPer>((const float*)logits + at, x);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        x[i] = kPer * ql + i < z.E ? load_logit(logits, z.f32, at + i) : -INFINITY;
    }
    if (!bias) one_zero(x);
    float top = 0.f, total = 1.f;
    if (!z.sigmoid && (scores || !z.normalize)) {
      top = x[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) top = fmaxf(top, x[i]);
      top = row_max_f(top);
      total = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) total += x[i] > -INFINITY ? expf(x[i] - top) : 0.f;
      total = row_sum_f(total);
    }
    float key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = x[i];
    if (scores) {
      const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        key[i] = x[i] > -INFINITY ? quick_key(x[i], b[i], z, top, inv) : -INFINITY;
    }
    bool unsure = false;
    if (z.groups > 1) {  // of 2^n lanes
      const int lanes = z.E / z.groups / kPer;
      float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        m2 = fmaxf(m2, fminf(m1, key[i]));
        m1 = fmaxf(m1, key[i]);
      }
      for (int o = 1; o < lanes; o <<= 1) {
        const float o1 = __shfl_xor(m1, o, kWave), o2 = __shfl_xor(m2, o, kWave);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
      // Ordered numbers of the sums, the group in the low four bits; lanes past
      // the experts have none.
      const float sum = m2 > -INFINITY ? sum_of_two(m1, m2) : m1;
      const int g = ql / lanes;
      uint32_t u = sum > -INFINITY && g < z.groups ? (ordered(sum) & ~15u) | (15u - g) : 0u;
      uint32_t last = 0;  // the topk_groups-th
      for (int k = 0; k < z.topk_groups; ++k) last = below(k, last, row_max_u(u - last));
      bool in = u != 0 && u >= last;
      // The least that a group chosen may have, and the most of one left out.
      const float error = sum_error(m1, m2, sum, z.sigmoid);
      const float least = -row_max_f(in ? error - sum : -INFINITY);
      const float most = row_max_f(u != 0 && !in ? sum + error : -INFINITY);
      unsure = most > -INFINITY && !(least > most);
      if (exact && __ballot(unsure)) {
        // fp64 sums of the two largest, from those that may be among them.
        float cut = m2 > -INFINITY ? m2 : m1;
        cut -= 2 * key_error(cut, z.sigmoid);
        uint32_t todo = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          todo |= (uint32_t)(key[i] > -INFINITY && key[i] >= cut) << i;
        double d1 = -INFINITY, d2 = -INFINITY;
        while (__ballot(todo != 0)) {
          const int at_i = __builtin_ctz(todo | 0x10000u);
          float xv = 0.f, bv = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (i == at_i) xv = x[i], bv = b[i];
          const double d = todo ? exact_key(xv, bv, z, top) : -INFINITY;
          d2 = max(d2, min(d1, d));
          d1 = max(d1, d);
          todo &= todo - 1;
        }
        for (int o = 1; o < lanes; o <<= 1) {
          const double o1 = __shfl_xor(d1, o, kWave), o2 = __shfl_xor(d2, o, kWave);
          d2 = max(min(d1, o1), max(d2, o2));
          d1 = max(d1, o1);
        }
        const double both = d2 > -INFINITY ? d1 + d2 : d1;
        int rank = 0;
        for (int j = 0; j < z.groups; ++j) {
          const double other = __shfl(both, (lane & 48) + j * lanes, kWave);
          rank += other > both || (other == both && j < g);
        }
        in = u != 0 && rank < z.topk_groups;
        unsure = unsure && !z.sigmoid && least < 0x1p-100f;  // (with softmax's sum, then)
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) key[i] = in && key[i] > -INFINITY ? (bias ? key[i] : x[i])
                                                                       : -INFINITY;
    }
    uint32_t u[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      u[i] = key[i] > -INFINITY
                 ? (ordered(key[i]) & ~kIndex) | (kIndex - (uint32_t)(kPer * ql + i))
                 : 0u;
    uint32_t mine = 0, best = 0;  // lane k of the row: the k-th
    for (int k = 0; k < z.topk + 2; ++k) {
      uint32_t m = u[0] - best;
#pragma unroll
      for (int i = 1; i < kPer; ++i) m = max(m, u[i] - best);
      best = below(k, best, row_max_u(m));
      if (ql == k) mine = best;
    }
    const uint32_t next = (uint32_t)dpp_move<0x101, 0xf>(0, (int)mine);  // row_shl:1
    int id = mine != 0 ? (int)(kIndex - (mine & kIndex)) : -1;
    float v = 0.f;
    if (id >= 0) v = load_logit(logits, z.f32, r * stride + id);
    bool near = false;  // the order of this one and the next is open
    if (loose && ql < z.topk && next != 0 && may_pass<kIndex>(next, mine, bias != nullptr, z)) {
      const int other = (int)(kIndex - (next & kIndex));
      near = v != load_logit(logits, z.f32, r * stride + other) || (bias && bias[id] != bias[other]);
    }
    if (!bias && z.groups > 1 && ql < z.topk && next != 0)
      unsure |= one_score<kIndex>(mine, next, z, top);
    // Where the first one left out equals the last one chosen, so must all that lie as
    // near to them.
    if (loose && __ballot(ql == z.topk - 1 && next != 0 && !near &&
                          may_pass<kIndex>(next, mine, bias != nullptr, z))) {
      const int from = (lane & 48) + z.topk - 1;
      const uint32_t last = (uint32_t)__shfl((int)mine, from, kWave);
      const float lv = __shfl(v, from, kWave);
      const int lid = __shfl(id, from, kWave);
      const float lb = lid >= 0 ? load_bias(bias, lid) : 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (u[i] != 0 && u[i] < last && may_pass<kIndex>(u[i], last, bias != nullptr, z))
          near |= x[i] != lv || b[i] != lb;
    }
    if (!exact) {
      unsure |= near;
    } else if (__ballot(near)) {
      // The topk + 2 that are lined up, by their exact keys.  What was not lined up
      // lies below the last of them: it has to lie below the topk-th key, too.
      float bv = 0.f;
      if (bias && id >= 0) bv = fminf(bias[id], FLT_MAX);
      const double d = id < 0 ? -INFINITY : bias ? exact_key(v, bv, z, top) : (double)v;
      int rank = 0;
      for (int j = 0; j < z.topk + 2; ++j) {
        const double other = __shfl(d, (lane & 48) + j, kWave);
        const int oid = __shfl(id, (lane & 48) + j, kWave);
        // (Lanes without an expert, -1, keep their order.)
        rank += other > d || (other == d && ((uint32_t)oid < (uint32_t)id ||
                                             (oid == id && j < ql)));
      }
      const float end = unordered(best | kIndex);
      unsure |= rank == z.topk - 1 && best != 0 &&
                d <= (double)end + (bias ? key_error(end, z.sigmoid) : 0.f);
      const int from = ql < z.topk + 2 ? rank : ql;  // a place of its own for every lane
      id = __builtin_amdgcn_ds_permute(((lane & 48) + from) * 4, id);
      v = __int_as_float(
          __builtin_amdgcn_ds_permute(((lane & 48) + from) * 4, __float_as_int(v)));
    }
    const bool here = ql < z.topk && id >= 0;
    if (!here) id = -1;
    float w;
    if (z.normalize) {
      const float low = here ? (z.sigmoid ? fminf(v, 0.f) : v) : -INFINITY;
      const float m = row_max_f(low);
      w = here ? expf(low - m) : 0.f;
      if (z.sigmoid) w /= 1.0f + expf(-fabsf(v));
      const float sum = row_sum_f(w);
      w = here ? w / sum : 0.f;
    } else {
      w = !here ? 0.f : z.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - top) / total;
    }
    const uint64_t open = __ballot(unsure && real);
    const bool again = (open >> (lane & 48) & 0xffff) != 0;
    if (real && !again && ql < z.topk) {
      ids[r * z.topk + ql] = id;
      weights[r * z.topk + ql] = w;
    }
    if (open) {
      for (int q = 0; q < 4; ++q)
        if (open >> (16 * q) & 0xffff)
          route_row<(kPer + 3) / 4, true>(logits, stride, bias, z, r0 + q, lane, true, ids,
                                          weights);
    }
  }
}

// A wave to a row.  wide: fp32, 64 kPer experts, 16-byte rows.
template <int kPer>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(
    const void* __restrict__ logits, int64_t stride, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, Sizes z, bool wide, const int32_t* __restrict__ psum_rank,
    int nsrc, int64_t rows, void* __restrict__ dx, int64_t dx_stride) {
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nv = valid_rows(psum_rank, nsrc, rows);
  const bool dense = !z.sigmoid && !z.normalize;  // every available expert has a gradient
  for (int64_t r = (int64_t)blockIdx.x * kWaves + wid; r < nv;
       r += (int64_t)gridDim.x * kWaves) {
    int id = -1;
    float g = 0.f, v = 0.f;
    if (lane < z.topk) {
      id = ids[r * z.topk + lane];
      g = dw[r * z.topk + lane];
    }
    float d[kPer];  // softmax's values, then the gradients
    float top = 0.f, total = 1.f, inv = 1.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) d[i] = 0.f;
    if (dense) {
      bool done = false;
      if constexpr (kPer % 4 == 0) {
        if (wide) {
          load_wide<kPer>((const float*)logits + r * stride + kPer * lane, d);
          done = true;
        }
      }
      if (!done) load_row<kPer>(logits, z, r * stride, lane, d);
      top = d[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) top = fmaxf(top, d[i]);
      top = wave_max_f(top);
      total = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        d[i] = d[i] > -INFINITY ? expf(d[i] - top) : 0.f;
        total += d[i];
      }
      total = wave_sum_f(total);
      inv = total > 0.f ? 1.0f / total : 0.f;
    }
    if (id < 0 || id >= z.E) id = -1;
    if (id >= 0) v = load_logit(logits, z.f32, r * stride + id);
    if (v == -INFINITY) id = -1;
    if (id < 0) g = 0.f;  // whatever it was
    const float w = weight_of(v, id, z, top, total);
    const float dot = wave_sum_f(w * g);
    float own;  // what the chosen experts get by themselves
    if (z.sigmoid) own = w * (1.0f / (1.0f + expf(v))) * (z.normalize ? g - dot : g);
    else own = w * (z.normalize ? g - dot : g);
    if (dense) {
      const float f = -inv * dot;
      if (fabsf(f) < INFINITY) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) d[i] *= f;
      } else {  // experts that are not available get 0 all the same
#pragma unroll
        for (int i = 0; i < kPer; ++i) d[i] = d[i] > 0.f ? d[i] * f : 0.f;
      }
    }
    for (int k = 0; k < z.topk; ++k) {
      const int e = __builtin_amdgcn_readlane(id, k);
      if (e < 0) continue;
      const float o = lane_value(own, k);
      const float add = lane == e / kPer ? o : 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (e % kPer == i) d[i] += add;  // the same branch for all lanes
    }
    if constexpr (kPer % 4 == 0) {
      if (wide) {
        v4f* to = reinterpret_cast<v4f*>((float*)dx + r * dx_stride + kPer * lane);
#pragma unroll
        for (int i = 0; i < kPer; i += 4) to[i / 4] = v4f{d[i], d[i + 1], d[i + 2], d[i + 3]};
        continue;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = kPer * lane + i;
      if (e >= z.E) continue;
      if (z.f32) ((float*)dx)[r * dx_stride + e] = d[i];
      else ((uint16_t*)dx)[r * dx_stride + e] = f32_to_bf16_rne(d[i]);
    }
  }
}

moe_status check(const void* logits, int64_t stride, moe_float_fmt fmt, moe_score score,
                 const int32_t* psum_recv_per_rank, int num_src_ranks, int64_t rows,
                 int num_experts, int topk) {
  if (rows < 0 || rows > (1LL << 30) || num_experts < 1 || num_experts > MOE_MAX_EXPERTS ||
      topk < 1 || topk > MOE_MAX_TOPK || topk > num_experts || stride < num_experts ||
      stride > (1LL << 30))
    return MOE_ERR_SHAPE;
  if (num_src_ranks < 0 || (psum_recv_per_rank && num_src_ranks == 0)) return MOE_ERR_SHAPE;
  if ((fmt != MOE_FLOAT_BF16 && fmt != MOE_FLOAT_F32) ||
      (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID))
    return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && !logits) return MOE_ERR_NULL;
  if ((uintptr_t)logits % (fmt == MOE_FLOAT_F32 ? 4 : 2)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

int64_t matrix_bytes(int64_t rows, int cols, int64_t stride, moe_float_fmt fmt) {
  return rows > 0 ? ((rows - 1) * stride + cols) * (fmt == MOE_FLOAT_F32 ? 4 : 2) : 0;
}

int64_t grid_of(int64_t rows) {
  const int64_t blocks = (rows + kWaves - 1) / kWaves;
  return blocks < 65536 ? blocks : 65536;  // grid-stride over the rest
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_router(const void* logits, int64_t logits_stride, moe_float_fmt fmt,
                                 const float* bias, moe_score score, int num_groups,
                                 int topk_groups, int normalize,
                                 const int32_t* psum_recv_per_rank, int num_src_ranks,
                                 int64_t rows, int num_experts, int topk, int32_t* topk_ids,
                                 float* topk_weights, void* stream) {
  const moe_status bad = check(logits, logits_stride, fmt, score, psum_recv_per_rank,
                               num_src_ranks, rows, num_experts, topk);
  if (bad != MOE_OK) return bad;
  if (num_groups < 1 || num_groups > kMaxGroups || num_experts % num_groups || topk_groups < 1 ||
      topk_groups > num_groups)
    return MOE_ERR_SHAPE;
  if (rows > 0 && (!topk_ids || !topk_weights)) return MOE_ERR_NULL;
  if ((uintptr_t)bias % 4 || (uintptr_t)topk_ids % 4 || (uintptr_t)topk_weights % 4)
    return MOE_ERR_ALIGNMENT;
  const int64_t in = matrix_bytes(rows, num_experts, logits_stride, fmt), out = rows * topk * 4;
  for (const void* o : {(const void*)topk_ids, (const void*)topk_weights})
    if (overlap(o, out, logits, in) || overlap(o, out, bias, num_experts * 4LL) ||
        overlap(o, out, psum_recv_per_rank, num_src_ranks * 4LL))
      return MOE_ERR_UNSUPPORTED;
  if (overlap(topk_ids, out, topk_weights, out)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const Sizes z = {num_experts,          topk, num_groups, topk_groups, fmt == MOE_FLOAT_F32,
                   score == MOE_SCORE_SIGMOID, normalize != 0};
  // Four rows to a wave, or one.  Groups are quick where each is 2^n lanes of
  // either.
  const int size = num_experts / num_groups;
  auto fits = [&](int per) {
    const int lanes = size / per;
    return num_groups == 1 || (size % per == 0 && (lanes & (lanes - 1)) == 0);
  };
  const int quad = num_experts <= 64 ? 4 : num_experts <= 128 ? 8 : 16;
  if (num_experts <= 256 && topk < 15 && fits(quad) && fits((quad + 3) / 4)) {
    const bool wide_loads = z.f32 && num_experts == 16 * quad && (uintptr_t)logits % 16 == 0 &&
                            (uintptr_t)bias % 16 == 0 && logits_stride % 4 == 0;
    const int64_t blocks = (rows + 4 * kWaves - 1) / (4 * kWaves);
    auto kern = quad == 4   ? router_quad_kernel<4>
                : quad == 8 ? router_quad_kernel<8>
                            : router_quad_kernel<16>;
    hipLaunchKernelGGL(kern, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0,
                       reinterpret_cast<hipStream_t>(stream), logits, logits_stride, bias, z,
                       wide_loads, psum_recv_per_rank, num_src_ranks, rows, topk_ids,
                       topk_weights);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
  }
  const int per = num_experts <= 64 ? 1 : num_experts <= 128 ? 2 : num_experts <= 256 ? 4
                  : num_experts <= 512 ? 8 : 16;
  const bool quick = fits(per);
  auto kern = per == 1   ? (quick ? router_kernel<1, true> : router_kernel<1, false>)
              : per == 2 ? (quick ? router_kernel<2, true> : router_kernel<2, false>)
              : per == 4 ? (quick ? router_kernel<4, true> : router_kernel<4, false>)
              : per == 8 ? (quick ? router_kernel<8, true> : router_kernel<8, false>)
                         : (quick ? router_kernel<16, true> : router_kernel<16, false>);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid_of(rows)), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), logits, logits_stride, bias, z,
                     psum_recv_per_rank, num_src_ranks, rows, topk_ids, topk_weights);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

extern "C" moe_status moe_router_backward(
    const void* logits, int64_t logits_stride, moe_float_fmt fmt, moe_score score, int normalize,
    const int32_t* topk_ids, const float* d_topk_weights, const int32_t* psum_recv_per_rank,
    int num_src_ranks, int64_t rows, int num_experts, int topk, void* d_logits,
    int64_t d_logits_stride, void* stream) {
  const moe_status bad = check(logits, logits_stride, fmt, score, psum_recv_per_rank,
                               num_src_ranks, rows, num_experts, topk);
  if (bad != MOE_OK) return bad;
  if (d_logits_stride < num_experts || d_logits_stride > (1LL << 30)) return MOE_ERR_SHAPE;
  if (rows > 0 && (!topk_ids || !d_topk_weights || !d_logits)) return MOE_ERR_NULL;
  if ((uintptr_t)d_logits % (fmt == MOE_FLOAT_F32 ? 4 : 2) || (uintptr_t)topk_ids % 4 ||
      (uintptr_t)d_topk_weights % 4)
    return MOE_ERR_ALIGNMENT;
  const int64_t in = matrix_bytes(rows, num_experts, logits_stride, fmt), slots = rows * topk * 4;
  const int64_t out = matrix_bytes(rows, num_experts, d_logits_stride, fmt);
  if (overlap(d_logits, out, logits, in) || overlap(d_logits, out, topk_ids, slots) ||
      overlap(d_logits, out, d_topk_weights, slots) ||
      overlap(d_logits, out, psum_recv_per_rank, num_src_ranks * 4LL))
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const Sizes z = {num_experts, topk, 1, 1, fmt == MOE_FLOAT_F32, score == MOE_SCORE_SIGMOID,
                   normalize != 0};
  auto kern = num_experts <= 64    ? router_backward_kernel<1>
              : num_experts <= 128 ? router_backward_kernel<2>
              : num_experts <= 256 ? router_backward_kernel<4>
              : num_experts <= 512 ? router_backward_kernel<8>
                                   : router_backward_kernel<16>;
  const bool wide = z.f32 && (num_experts == 256 || num_experts == 512 || num_experts == 1024) &&
                    (uintptr_t)logits % 16 == 0 && (uintptr_t)d_logits % 16 == 0 &&
                    logits_stride % 4 == 0 && d_logits_stride % 4 == 0;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid_of(rows)), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), logits, logits_stride, topk_ids,
                     d_topk_weights, z, wide, psum_recv_per_rank, num_src_ranks, rows, d_logits,
                     d_logits_stride);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
