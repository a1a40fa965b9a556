// moe_adamw: one AdamW step with decoupled weight decay over many tensors,
// with fp32 or 8-bit states.
//
//   g = grad * grad_scale
//   m = m * b1 + g * (1 - b1),   v = v * b2 + g^2 * (1 - b2)
//   master -= lr * (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + wd * master)
//
// 8-bit states: groups of 128 consecutive values as E4M3 codes and an fp32
// scale.  The second moment is kept as its root r = sqrt(v): the codes cover
// 448 / 2^-9 = 2.3e5 between the largest and the smallest value of a group,
// for r that is 5e10 in v.  The codes are decided in fp32 with every
// operation rounded in the order above (no contraction), so they are the ones
// that the same sequence of elementwise fp32 operations gives.
//
// Codes lie 6 to 12 % apart.  A state whose beta is near 1 moves by less than
// half of that in a step, and the nearest code would be the one it has, step
// after step: it would follow its group's largest value and nothing else.  Such
// a state (beta > 31/32) goes to one of its two neighbouring codes instead, to
// the nearer one as much more often as it is nearer, so that small moves come
// through on average.  The choice is taken from a hash of the new states and the
// step's number: equal calls still give equal codes.  Measured (roots against
// those of fp32 states, half of each group's gradients falling tenfold; median
// some lives of the average later): beta 0.999, 5.5 times too large with the
// nearest codes, 0.96 with these; 0.99, 7.7 and 0.99; 0.98, 1.8 and 0.99.  Up to
// 0.97 the gradients' own noise carries states from code to code, and the
// nearest ones stay closer: 0.96, 5th to 95th percentile 0.87 to 1.12 against
// 0.83 to 1.21.  The hash costs 10 % with one state's codes chosen by it, 15 % with
// both (354M values: 1000, 1100 and 1150 us).
//
// HBM-bound: everything is read once and written once, past the caches.  A
// workgroup takes 1024 or 2048 values of one tensor; the list of tensors
// travels in the kernel's arguments (nothing is copied to the device), up to
// kMaxTensors per launch.  Each lane owns 4 consecutive values, so that every
// access of a wave is one contiguous run (8 per lane, in two pieces for the
// fp32 arrays: 566 us against 527 at 100M values with fp32 states), and a group
// of 128 is 32 lanes.  354M values with 8-bit states take 1000 us, 5.7 TB/s;
// 100M with fp32 states 460 us, 6.1 TB/s (with accesses through the caches
// 1110 and 527).
#include <float.h>
#include <stdlib.h>

#include <algorithm>

#include "lds_dma.hpp"

// Each operation rounded by itself: plain operators under this pragma (the
// header's __fmul_rn and __fadd_rn may still be joined into one fma).
#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;                              // consecutive values per lane
constexpr int kPart = kThreads * kVec;
// Parts per workgroup.  With 8-bit states two, whose loads are asked for
// together (354M values: 1015 us against 1100 with one), with fp32 ones one
// (100M: 463 against 492 with two).
__host__ __device__ constexpr int parts(int state_fmt) {
  return state_fmt == MOE_STATE_FP8 ? 2 : 1;
}
__host__ __device__ constexpr int chunk(int state_fmt) { return kPart * parts(state_fmt); }
// Values of a tensor: a launch has fewer than 2^32 threads.
constexpr int64_t kMaxNumel = 1LL << 33;
constexpr int kMaxTensors = 32;                      // per launch (kernel arguments: 4 KB)
constexpr float kFp8Max = 448.f, kCodeMin = 0x1p-9f, kAmaxFloor = 0x1p-100f;
static_assert(MOE_STATE_GROUP == 128 && kPart % MOE_STATE_GROUP == 0, "groups fill parts");

struct Batch {
  moe_adamw_tensor t[kMaxTensors];
  int64_t first[kMaxTensors + 1];  // first workgroup of each tensor
  int count;
};
static_assert(sizeof(Batch) <= 3584, "kernel argument size");

struct Hyper {
  double beta1, beta2;
  float b1, one_b1, b2, one_b2, eps, wd;
  bool dither_m, dither_r;  // codes chosen by hash, not the nearest
};
constexpr double kNearestBeta = 31.0 / 32;  // up to it a state gets its nearest code

// b^t in fp64 by repeated squaring (t >= 1 is the step's number).
__device__ __forceinline__ double pow_int(double b, int64_t t) {
  double r = 1.0;
  for (uint64_t n = t > 0 ? (uint64_t)t : 0; n; n >>= 1) {
    if (n & 1) r *= b;
    b *= b;
  }
  return r;
}

struct Step {
  float rc1, rr2, lr, gs;  // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t)
};

// New m and v (and r = sqrt(v)), each operation rounded by itself.  The step
// takes them with one reciprocal and two products where the formula has three
// quotients and another root: a few fp32 steps off the update, which moves
// the master by far less than its own last rounding does.  (The reciprocal's
// argument is normal or 0: the root of any positive fp32 value is at least 2^-75,
// and an eps below the normal range is refused; the reciprocal of one would be
// infinite.)
__device__ __forceinline__ void update(const Hyper& h, const Step& st, float grad, float& p,
                                       float& m, float& v, float& r) {
  const float g = grad * st.gs;
  m = m * h.b1 + g * h.one_b1;
  v = v * h.b2 + (g * g) * h.one_b2;
  r = sqrtf(v);
  const float u = (m * st.rc1) * __builtin_amdgcn_rcpf(r * st.rr2 + h.eps);
  p = p - (u + p * h.wd) * st.lr;
}

// Largest magnitude of the 32 lanes that hold a group, not below the floor.
__device__ __forceinline__ float group_amax(const float (&x)[kVec]) {
  float a = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < kVec; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor(a, o, kWave));
  return a;
}

// 32 bits that look random, from an element's new states and the step's number:
// products with odd numbers (2^32 times the fractional parts of the golden ratio
// and of the roots of 2 and 3) and shifted sums.  The upper 20 bits are for m,
// the lower 20 for r.
__device__ __forceinline__ uint32_t dither_bits(float m, float r, uint32_t step) {
  uint32_t h = __float_as_uint(m) ^ __builtin_rotateleft32(__float_as_uint(r), 11);
  h = h * 0x9e3779b9u + step * 0xbb67ae85u;
  h = (h ^ (h >> 16)) * 0x9e3779b9u;
  h = (h ^ (h >> 15)) * 0x6a09e667u;
  return h ^ (h >> 16);
}

// q (in units of the scale) to one of its two neighbouring codes: 20 random bits
// are added below the last bit that a code keeps, and cut off.  Below 2^-6 codes
// are 2^-9 apart: so are the ones from 2^-6 to 2^-5, where q is moved to and back.
__device__ __forceinline__ float to_neighbour(float q, uint32_t bits20) {
  const float a = fabsf(q);
  const bool low = a < 0x1p-6f;
  float t = low ? a + 0x1p-6f : a;
  t = __uint_as_float((__float_as_uint(t) + bits20) & 0xfff00000u);
  if (low) t -= 0x1p-6f;
  return a <= kFp8Max ? copysignf(t, q) : q;  // the largest, rounded up; NaN
}

// Codes of x and their group's scale: the nearest, or with `dither` chosen by
// the 20 bits of u at `shift`.
template <bool kPositive, bool kDither>
__device__ __forceinline__ uint32_t encode(const float (&x)[kVec], float& scale, bool dither,
                                           const uint32_t (&u)[kVec], int shift) {
  const float amax = group_amax(x);
  scale = amax * (1.f / kFp8Max);
  const float inv = (1.f / amax) * kFp8Max;
  float q[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    q[i] = x[i] * inv;
    if (kPositive && x[i] > 0.f) q[i] = fmaxf(q[i], kCodeMin);
    if (kDither && dither) q[i] = to_neighbour(q[i], u[i] >> shift & 0xfffffu);
  }
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
}

__device__ __forceinline__ void decode(uint32_t c, float scale, float (&x)[kVec]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
  const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  const float y[kVec] = {a[0], a[1], b[0], b[1]};
#pragma unroll
  for (int i = 0; i < kVec; ++i) x[i] = y[i] * scale;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// n (1..kVec) consecutive values at p + i; whole vectors where n == kVec (the
// base is 16-byte aligned and i a multiple of kVec).
__device__ __forceinline__ void load_f32(const float* p, int64_t i, int n, float (&x)[kVec]) {
  if (n == kVec) {
    const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i));
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = a[j];
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = j < n ? p[i + j] : 0.f;
  }
}
__device__ __forceinline__ void store_f32(float* p, int64_t i, int n, const float (&x)[kVec]) {
  if (n == kVec) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n) p[i + j] = x[j];
  }
}
__device__ __forceinline__ void load_bf16(const uint16_t* p, int64_t i, int n, float (&x)[kVec]) {
  if (n == kVec) {
    const u32x2 a = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + i));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x[2 * j] = __uint_as_float(a[j] << 16);
      x[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = j < n ? bf16_to_f32(p[i + j]) : 0.f;
  }
}
__device__ __forceinline__ void store_bf16(uint16_t* p, int64_t i, int n, const float (&x)[kVec]) {
  if (n == kVec) {
    __builtin_nontemporal_store(u32x2{pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])},
                                reinterpret_cast<u32x2*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n) p[i + j] = f32_to_bf16_rne(x[j]);
  }
}
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int n) {
  if (n == kVec) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p + i));
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    if (j < n) w |= (uint32_t)p[i + j] << (8 * j);
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int n, uint32_t c) {
  if (n == kVec) {
    __builtin_nontemporal_store(c, reinterpret_cast<uint32_t*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n) p[i + j] = (uint8_t)(c >> (8 * j));
  }
}

template <bool kGradF32, bool kFp8, bool kDither>
__device__ __forceinline__ void run_chunk(const moe_adamw_tensor& t, int64_t base,
                                          const Hyper& h, const Step& st, uint32_t step) {
  constexpr int kParts = parts(kFp8 ? MOE_STATE_FP8 : MOE_STATE_F32);
  // Values past the end are 0 and stay so; their lanes take part in the
  // group's maximum.
  float g[kParts][kVec] = {}, p[kParts][kVec] = {}, m[kParts][kVec] = {}, v[kParts][kVec] = {};
  int n[kParts];
#pragma unroll
  for (int u = 0; u < kParts; ++u) {
    const int64_t i = base + u * kPart + threadIdx.x * kVec;
    n[u] = (int)max((int64_t)0, min((int64_t)kVec, t.numel - i));
    if (n[u] <= 0) continue;
    if (kGradF32) load_f32((const float*)t.grad, i, n[u], g[u]);
    else load_bf16((const uint16_t*)t.grad, i, n[u], g[u]);
    load_f32(t.master, i, n[u], p[u]);
    if constexpr (kFp8) {
      const uint32_t cm = load_codes((const uint8_t*)t.m, i, n[u]);
      const uint32_t cv = load_codes((const uint8_t*)t.v, i, n[u]);
      decode(cm, t.m_scale[i / MOE_STATE_GROUP], m[u]);
      decode(cv, t.v_scale[i / MOE_STATE_GROUP], v[u]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[u][j] = v[u][j] * v[u][j];
    } else {
      load_f32((const float*)t.m, i, n[u], m[u]);
      load_f32((const float*)t.v, i, n[u], v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kParts; ++u) {
    const int64_t i = base + u * kPart + threadIdx.x * kVec;
    float r[kVec] = {};
    if (n[u] > 0) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) update(h, st, g[u][j], p[u][j], m[u][j], v[u][j], r[j]);
      store_f32(t.master, i, n[u], p[u]);
      if (t.param) store_bf16((uint16_t*)t.param, i, n[u], p[u]);
    }
    if constexpr (kFp8) {
      float sm, sv;
      uint32_t bits[kVec] = {};
      if constexpr (kDither) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) bits[j] = dither_bits(m[u][j], r[j], step);
      }
      const uint32_t cm = encode<false, kDither>(m[u], sm, h.dither_m, bits, 12);
      const uint32_t cv = encode<true, kDither>(r, sv, h.dither_r, bits, 0);
      if (n[u] > 0) {
        store_codes((uint8_t*)t.m, i, n[u], cm);
        store_codes((uint8_t*)t.v, i, n[u], cv);
        if ((threadIdx.x & 31) == 0) {
          t.m_scale[i / MOE_STATE_GROUP] = sm;
          t.v_scale[i / MOE_STATE_GROUP] = sv;
        }
      }
    } else if (n[u] > 0) {
      store_f32((float*)t.m, i, n[u], m[u]);
      store_f32((float*)t.v, i, n[u], v[u]);
    }
  }
}

// kDither: codes of one state at least are chosen by hash (a kernel of its own:
// in one, the nearest ones cost 1 % more).
template <bool kDither>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Batch b, const Hyper h,
                                                         const int64_t* __restrict__ step,
                                                         const float* __restrict__ lr,
                                                         const float* __restrict__ grad_scale) {
  int q = 0;
  while (q + 1 < b.count && (int64_t)blockIdx.x >= b.first[q + 1]) ++q;  // uniform
  const moe_adamw_tensor& t = b.t[q];
  const int64_t base = ((int64_t)blockIdx.x - b.first[q]) * chunk(t.state_fmt);
  const int64_t n = *step;
  const float c1 = (float)(1.0 - pow_int(h.beta1, n)), c2 = (float)(1.0 - pow_int(h.beta2, n));
  const Step st = {1.f / c1, 1.f / sqrtf(c2), *lr, grad_scale ? *grad_scale : 1.f};
  if (t.state_fmt == MOE_STATE_FP8) {
    if (t.grad_fmt == MOE_GRAD_F32) run_chunk<true, true, kDither>(t, base, h, st, (uint32_t)n);
    else run_chunk<false, true, kDither>(t, base, h, st, (uint32_t)n);
  } else {
    if (t.grad_fmt == MOE_GRAD_F32) run_chunk<true, false, kDither>(t, base, h, st, (uint32_t)n);
    else run_chunk<false, false, kDither>(t, base, h, st, (uint32_t)n);
  }
}

// One tensor's arguments; MOE_OK also for an empty one.
moe_status check_tensor(const moe_adamw_tensor& t) {
  if (t.numel < 0 || t.numel > kMaxNumel) return MOE_ERR_SHAPE;
  if ((t.grad_fmt != MOE_GRAD_BF16 && t.grad_fmt != MOE_GRAD_F32) ||
      (t.state_fmt != MOE_STATE_F32 && t.state_fmt != MOE_STATE_FP8))
    return MOE_ERR_UNSUPPORTED;
  if (t.numel == 0) return MOE_OK;
  if (!t.master || !t.grad || !t.m || !t.v) return MOE_ERR_NULL;
  if (t.state_fmt == MOE_STATE_FP8 && (!t.m_scale || !t.v_scale)) return MOE_ERR_NULL;
  if (((uintptr_t)t.master % 16) || ((uintptr_t)t.grad % 16) || ((uintptr_t)t.m % 16) ||
      ((uintptr_t)t.v % 16) || ((uintptr_t)t.param % 16))
    return MOE_ERR_ALIGNMENT;
  if (t.state_fmt == MOE_STATE_FP8 && (((uintptr_t)t.m_scale % 4) || ((uintptr_t)t.v_scale % 4)))
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Memory that a call reads or writes.
struct Range {
  uintptr_t begin, end;
  bool written;
};

// MOE_OK if no array that the call writes shares memory with another that it
// reads or writes: two updates of one value would race.  Sorted by their
// begins, a range overlaps an earlier one if it begins below the furthest end
// so far.  (On the host, per call: 0.15 us for six tensors with fp32 states, 4 us
// for 75 with 8-bit ones.)
moe_status check_apart(const moe_adamw_tensor* tensors, int num_tensors, const int64_t* step,
                       const float* lr, const float* grad_scale) {
  constexpr int kScalars = 3, kArrays = 7, kFew = 32;
  Range few[kScalars + kArrays * kFew];
  Range* all = few;
  if (num_tensors > kFew) {
    all = (Range*)malloc((kScalars + kArrays * (size_t)num_tensors) * sizeof(Range));
    if (!all) return MOE_ERR_LAUNCH;
  }
  size_t n = 0;
  auto add = [&](const void* p, int64_t bytes, bool written) {
    if (p) all[n++] = {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written};
  };
  add(step, 8, false);
  add(lr, 4, false);
  add(grad_scale, 4, false);
  for (int i = 0; i < num_tensors; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.numel == 0) continue;
    const bool fp8 = t.state_fmt == MOE_STATE_FP8;
    const int64_t state = t.numel * (fp8 ? 1 : 4);
    add(t.master, t.numel * 4, true);
    add(t.grad, t.numel * (t.grad_fmt == MOE_GRAD_F32 ? 4 : 2), false);
    add(t.m, state, true);
    add(t.v, state, true);
    add(t.param, t.numel * 2, true);
    if (fp8) {
      const int64_t scales = (t.numel + MOE_STATE_GROUP - 1) / MOE_STATE_GROUP * 4;
      add(t.m_scale, scales, true);
      add(t.v_scale, scales, true);
    }
  }
  if (n <= 64) {  // mostly in order: allocations of one list follow each other
    for (size_t i = 1; i < n; ++i) {
      const Range r = all[i];
      size_t j = i;
      for (; j > 0 && all[j - 1].begin > r.begin; --j) all[j] = all[j - 1];
      all[j] = r;
    }
  } else {
    std::sort(all, all + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  }
  uintptr_t end = 0, end_written = 0;  // the furthest of all, of the written ones
  bool apart = true;
  for (size_t i = 0; i < n && apart; ++i) {
    const Range& r = all[i];
    apart = r.begin >= (r.written ? end : end_written);
    end = std::max(end, r.end);
    if (r.written) end_written = std::max(end_written, r.end);
  }
  if (all != few) free(all);
  return apart ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_adamw(const moe_adamw_tensor* tensors, int num_tensors,
                                const int64_t* step, const float* lr, const float* grad_scale,
                                double beta1, double beta2, double eps, double weight_decay,
                                void* stream) {
  if (num_tensors < 0) return MOE_ERR_SHAPE;
  // Written so that NaN fails too.
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
      !(eps >= 0.0 && eps <= 3.4e38) || !(weight_decay >= 0.0 && weight_decay <= 3.4e38))
    return MOE_ERR_SHAPE;
  if (eps > 0.0 && (float)eps < FLT_MIN) return MOE_ERR_SHAPE;
  if (!step || !lr || (num_tensors > 0 && !tensors)) return MOE_ERR_NULL;
  if (((uintptr_t)step % 8) || ((uintptr_t)lr % 4) || ((uintptr_t)grad_scale % 4))
    return MOE_ERR_ALIGNMENT;
  for (int i = 0; i < num_tensors; ++i) {
    const moe_status s = check_tensor(tensors[i]);
    if (s != MOE_OK) return s;
  }
  const moe_status apart = check_apart(tensors, num_tensors, step, lr, grad_scale);
  if (apart != MOE_OK) return apart;
  const Hyper h = {beta1, beta2, (float)beta1, (float)(1.0 - beta1), (float)beta2,
                   (float)(1.0 - beta2), (float)eps, (float)weight_decay,
                   beta1 > kNearestBeta, beta2 > kNearestBeta};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const auto kern = h.dither_m || h.dither_r ? adamw_kernel<true> : adamw_kernel<false>;
  for (int i = 0; i < num_tensors;) {
    Batch b;
    b.count = 0;
    b.first[0] = 0;
    int64_t blocks = 0;
    constexpr int64_t kMaxBlocks = kMaxNumel / kPart;  // one tensor has no more
    for (; i < num_tensors && b.count < kMaxTensors; ++i) {
      const int c = chunk(tensors[i].state_fmt);
      const int64_t n = (tensors[i].numel + c - 1) / c;
      if (n == 0) continue;
      if (b.count > 0 && blocks + n > kMaxBlocks) break;
      b.t[b.count] = tensors[i];
      blocks += n;
      b.first[++b.count] = blocks;
    }
    if (b.count == 0) break;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, b, h, step, lr,
                       grad_scale);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH;
  }
  return MOE_OK;
}
