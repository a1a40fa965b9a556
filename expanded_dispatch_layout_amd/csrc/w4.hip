// moe_grouped_gemm_w4: grouped products of bf16 rows with 4-bit expert weights.
//
//   out[m, j] = sum over groups g of s[e, j, g] * sum_{t in g} a[m, t] q[e, j, t]
//
// int4: q in [-8, 7], bf16 scales; MXFP4: q an E2M1 value, s = 2^(byte - 127).
//
// One workgroup of four waves per item (expert, up to 16 of its rows, 64
// columns); the waves take every fourth 128-deep block of the reduction, straight
// from memory into registers, and their sums meet in LDS in the waves' order.
//
// Codes to bf16.  A lane loads 16 bytes, 32 codes along the reduction, of one
// column; a 4 x 4 exchange between the four 16-lane rows of the wave then leaves each
// of its four words in the MFMA that covers the word's 32 deep group.  MXFP4:
// v_cvt_scalef32_pk_bf16_fp4 makes two values with their scale, exactly (a
// normal bf16 number for bytes 2..252).  int4: with u = q + 8, the bits 0x4180 | u << 3
// are the bf16 value 16 + u; the product starts from -24 * (the rows' own sum)
// instead of 0, one MFMA with a constant operand for all the columns, and is
// scaled in fp32 once its group is complete.
#include "gemm_backward.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kRows = 16, kCols = 64, kTiles = kCols / 16;
constexpr int BK = 128;

// 4 x 4 words between the wave's 16-lane rows: word i of row r <-> word r of
// row i.
__device__ __forceinline__ void exchange(u32x4& d) {
  uint32_t x[4] = {d[0], d[1], d[2], d[3]};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto h = __builtin_amdgcn_permlane32_swap(x[i], x[i + 2], false, false);
    x[i] = h[0];
    x[i + 2] = h[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto h = __builtin_amdgcn_permlane16_swap(x[i], x[i + 1], false, false);
    x[i] = h[0];
    x[i + 1] = h[1];
  }
  d = u32x4{x[0], x[1], x[2], x[3]};
}

// 8 E2M1 codes times a power of two.
__device__ __forceinline__ bf16x8 fp4_values(uint32_t d, float scale) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3));
  return __builtin_bit_cast(bf16x8, r);
}
// 8 int4 codes q as 24 + q.
__device__ __forceinline__ bf16x8 int4_values(uint32_t d) {
  const uint32_t lo = ((d << 3) & 0x78787878u) ^ 0xc0c0c0c0u;  // codes 0, 2, 4, 6
  const uint32_t hi = ((d >> 1) & 0x78787878u) ^ 0xc0c0c0c0u;  // codes 1, 3, 5, 7
  u32x4 r;
  r[0] = __builtin_amdgcn_perm(hi, lo, 0x0c040c00u) | 0x41004100u;
  r[1] = __builtin_amdgcn_perm(hi, lo, 0x0c050c01u) | 0x41004100u;
  r[2] = __builtin_amdgcn_perm(hi, lo, 0x0c060c02u) | 0x41004100u;
  r[3] = __builtin_amdgcn_perm(hi, lo, 0x0c070c03u) | 0x41004100u;
  return __builtin_bit_cast(bf16x8, r);
}

// kGroup 0: MXFP4; otherwise int4 with scales per 32, 64 or 128.
template <int kGroup>
struct Scales {  // of one column's 128-deep block
  static constexpr int kPer = BK / (kGroup ? kGroup : 32);
  uint32_t w[2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (kGroup == 0 || kGroup == 64) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kGroup == 128) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      w[0] = v[0];
      w[1] = v[1];
    }
  }
  __device__ __forceinline__ float get(int i) const {  // group i
    if constexpr (kGroup == 0) return __uint_as_float((w[0] >> (8 * i) & 0xffu) << 23);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};

template <int kGroup>
__global__ __launch_bounds__(kThreads) void w4_kernel(
    const uint8_t* __restrict__ a, const uint8_t* __restrict__ w, const uint8_t* __restrict__ sc,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, uint16_t* __restrict__ out) {
  constexpr bool kFp4 = kGroup == 0;
  constexpr int kScBytes = kFp4 ? 4 : 2 * Scales<kGroup>::kPer;  // per column and block
  __shared__ v4f lds[kWaves][kRows][kCols / 4 + 1];
  __shared__ int gp[MOE_MAX_EXPERTS + 1];  // prefix of 16-row groups per expert
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nrows = min((int64_t)status[0], capacity);
  auto expert_rows = [&](int e, int64_t& st, int64_t& en) __attribute__((always_inline)) {
    st = e ? max(0, align_up_i(psum[e - 1], align)) : 0;
    en = min((int64_t)psum[e], nrows);
  };
  if (wid == 0) {
    int sum = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      int ng = 0;
      if (e < E) {
        int64_t st, en;
        expert_rows(e, st, en);
        ng = en > st ? (int)((en - st + kRows - 1) / kRows) : 0;
      }
      const int incl = wave_incl_scan_i(ng);
      if (e < E) gp[e] = sum + incl - ng;
      sum += __shfl(incl, 63, 64);
    }
    if (lane == 0) gp[E] = sum;
  }
  __syncthreads();
  const int NT = n / kCols, KB = k / BK;
  const uint32_t nitems = (uint32_t)__builtin_amdgcn_readfirstlane(gp[E]) * (uint32_t)NT;
  for (uint32_t base = 0; base < nitems; base += gridDim.x) {
    const uint32_t item = round_item(base, nitems);
    if (item >= nitems) break;
    const int q = (int)(item / (uint32_t)NT);
    int lo = 0, hi = E - 1;  // last e with gp[e] <= q
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (gp[mid] <= q) lo = mid;
      else hi = mid - 1;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    const int g0 = __builtin_amdgcn_readfirstlane(gp[e]);
    const int ge = __builtin_amdgcn_readfirstlane(gp[e + 1]) - g0;
    const int local = (int)(item - (uint32_t)NT * (uint32_t)g0);
    const int n0 = local / ge * kCols;
    int64_t st, en;
    expert_rows(e, st, en);
    const int64_t m0 = st + (int64_t)(local % ge) * kRows;
    const int live = (int)min((int64_t)kRows, en - m0);

    const int c = lane & 15, qd = lane >> 4;
    const bool row = c < live;
    const uint8_t* ap = a + ((m0 + c) * k + 8 * qd) * 2;
    const uint8_t* wp = w + ((int64_t)e * n + n0 + c) * (k / 2) + 16 * qd;
    const uint8_t* sp = sc + ((int64_t)e * n + n0 + c) * (int64_t)KB * kScBytes;
    v4f acc[kTiles] = {};
    for (int kb = wid; kb < KB; kb += kWaves) {
      u32x4 av[4], wv[kTiles];
      Scales<kGroup> s[kTiles];
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        wv[j] = *reinterpret_cast<const u32x4*>(wp + (int64_t)j * 16 * (k / 2) + kb * (BK / 2));
        s[j].load(sp + ((int64_t)j * 16 * KB + kb) * kScBytes);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        av[i] = u32x4{0, 0, 0, 0};
        if (row) av[i] = *reinterpret_cast<const u32x4*>(ap + (kb * BK + 32 * i) * 2);
      }
#pragma unroll
      for (int j = 0; j < kTiles; ++j) exchange(wv[j]);
      v4f part[kTiles];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8 x = __builtin_bit_cast(bf16x8, av[i]);
        if constexpr (kFp4) {
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, fp4_values(wv[j][i], s[j].get(i)),
                                                             acc[j], 0, 0, 0);
        } else {
          constexpr int kSteps = kGroup / 32;  // MFMAs per group
          const u32x4 m24 = {0xc1c0c1c0u, 0xc1c0c1c0u, 0xc1c0c1c0u, 0xc1c0c1c0u};  // -24
          v4f off = {0.f, 0.f, 0.f, 0.f};
          off = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, __builtin_bit_cast(bf16x8, m24), off,
                                                        0, 0, 0);
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            const v4f from = i % kSteps == 0 ? off : part[j] + off;
            part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, int4_values(wv[j][i]), from, 0,
                                                              0, 0);
            if (i % kSteps == kSteps - 1) acc[j] += part[j] * s[j].get(i / kSteps);
          }
        }
      }
    }
    // lane: rows 4 qd + 0..3 of column 16 j + c
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        reinterpret_cast<float*>(lds[wid][4 * qd + r])[16 * j + c] = acc[j][r];
    __syncthreads();
    const int orow = threadIdx.x >> 4, oc = threadIdx.x & 15;
    v4f v = lds[0][orow][oc];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v += lds[i][orow][oc];
    if (orow < live) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *reinterpret_cast<u32x2*>(out + (m0 + orow) * n + n0 + 4 * oc) =
          u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
    }
    __syncthreads();  // the partial sums have been read
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_grouped_gemm_w4(const void* a, const void* w, const void* w_scale,
                                          moe_w4_fmt fmt, int group, const int32_t* psum,
                                          const int32_t* status, int64_t capacity, int n, int k,
                                          int num_experts, int align, void* out, void* stream) {
  if (capacity < 0 || capacity > (1LL << 30) || n <= 0 || k <= 0 || n % 128 || k % BK ||
      num_experts < 1 || num_experts > MOE_MAX_EXPERTS)
    return MOE_ERR_SHAPE;
  if (align < MOE_MIN_ALIGN || align > MOE_MAX_ALIGN || (align & (align - 1)))
    return MOE_ERR_UNSUPPORTED;
  if (capacity % align != 0) return MOE_ERR_SHAPE;
  if (fmt == MOE_W4_INT4 ? group != 32 && group != 64 && group != 128
                         : fmt != MOE_W4_MXFP4 || group != 32)
    return MOE_ERR_UNSUPPORTED;
  if (n / 64 > kMaxBlocks64 || k / 64 > kMaxBlocks64) return MOE_ERR_UNSUPPORTED;
  if (!psum || !status || !w || !w_scale) return MOE_ERR_NULL;
  if (capacity > 0 && (!a || !out)) return MOE_ERR_NULL;
  if ((uintptr_t)a % 16 || (uintptr_t)w % 16 || (uintptr_t)out % 16 || (uintptr_t)w_scale % 16)
    return MOE_ERR_ALIGNMENT;
  if (capacity == 0) return MOE_OK;
  const int64_t bytes = capacity * n * 2, cols = (int64_t)num_experts * n;
  if (overlap(out, bytes, a, capacity * k * 2) || overlap(out, bytes, w, cols * (k / 2)) ||
      overlap(out, bytes, w_scale, cols * (k / group) * (fmt == MOE_W4_INT4 ? 2 : 1)) ||
      overlap(out, bytes, psum, num_experts * 4LL) || overlap(out, bytes, status, 8))
    return MOE_ERR_UNSUPPORTED;
  int64_t grid = ((capacity + kRows - 1) / kRows + num_experts) * (int64_t)(n / kCols);
  if (grid > 2 * device_cus()) grid = 2 * device_cus();
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  auto kern = fmt == MOE_W4_MXFP4 ? w4_kernel<0>
              : group == 32       ? w4_kernel<32>
              : group == 64       ? w4_kernel<64>
                                  : w4_kernel<128>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), (const uint8_t*)a, (const uint8_t*)w,
                     (const uint8_t*)w_scale, psum, status, capacity, n, k, num_experts, align,
                     (uint16_t*)out);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
