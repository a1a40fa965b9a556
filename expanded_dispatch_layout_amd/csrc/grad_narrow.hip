// The grouped products' gradients where the 256 x 256 tiles of dgrad.hip and
// wgrad.hip are too few to fill the CUs: 64 x 64 tiles, the reduction split
// over the eight waves of a workgroup.  Bound by latency: launch, layout, a few
// rounds of loads, the joining of the waves (140 rows, 6 x 896 x 640: 6.8 us,
// below the 7.4 that a call takes to issue).
//
//  - A wave takes every eighth 32-deep stage of the reduction.  Its stages are
//    its own: it loads them HBM -> LDS into its own 16 KB, two stages or three, and
//    waits for its own loads only, so there is no barrier in the loop.
//  - The eight partial tiles (fp32) meet in LDS, each in its wave's own slots,
//    and are summed in the waves' order: equal calls give equal bits.
//  - Each stage is 64 MFMA-rows and 64 MFMA-columns by 32: 16
//    v_mfma_f32_16x16x32_bf16 on fragments read through ds_read_b64_tr_b16
//    where the reduction runs along the staged rows (w, and both operands of
//    the weight gradient), and as 16-byte pieces where it runs along the
//    columns (dy of the input gradient).
#include <type_traits>

#include "gemm_backward.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512, kWaves = 8;
constexpr int T = kNarrowTile;            // 64
constexpr int kStep = 32;
constexpr int kOpBytes = 4096;            // one operand of a stage: 32 x 64 bf16
constexpr int kWaveBytes = T * T * 4;     // slots of stages; later one fp32 64 x 64 tile

// Row-staged operand (reduction along the rows): 32 rows of 128 bytes.  Four
// 32-byte pieces per row, XOR-swizzled by row so that the 8 rows that half a
// wave reads at once fall on different banks (two rows make 256 bytes).
__device__ __forceinline__ int row_key(int row) {
  return ((row >> 1) & 1) | (((row >> 3) & 1) << 1);
}
// Column-staged operand (reduction along the columns): 64 rows of 64 bytes,
// four 16-byte chunks per row, XOR-swizzled by row / 4 -> 0, 2, 3, 1: no bank
// conflicts between 16 consecutive lanes, nor between lanes 0-3 and 12-15 of
// one 16-lane group and 4-11 of the next.
__device__ __forceinline__ int col_key(int row) { return 0x78 >> (2 * ((row >> 2) & 3)) & 3; }

// Fragment addresses of this lane within an operand: tile i is at ^ (i << 5)
// (row-staged) or + i * 1024 (column-staged).
__device__ __forceinline__ uint32_t row_lane(int lane) {
  const int row = 8 * (lane >> 4) + ((lane & 15) >> 2), q = lane & 3;
  return (uint32_t)(row * 128 + row_key(row) * 32 + (q >> 1) * 16 + (q & 1) * 8);
}
__device__ __forceinline__ uint32_t col_lane(int lane) {
  const int row = lane & 15;
  return (uint32_t)(row * 64 + (((lane >> 4) ^ col_key(row)) << 4));
}

// Loads q = 0..3 of a row-staged operand: rows 8 q + lane / 8, from a matrix
// whose row 0 and column 0 are at src (pitch ld bytes); rows >= nr are zeros.
__device__ __forceinline__ void load_rows(const uint8_t* src, int64_t ld, int nr, uint32_t lds,
                                          int lane) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = 8 * q + (lane >> 3);
    const uint8_t* p = src + row * ld + (((lane & 7) ^ (row_key(row) << 1)) << 4);
    dma16_ptr(row < nr ? p : zero_chunk(), lds + q * 1024);
  }
}
// Loads q < kQ of a column-staged operand: rows 16 q + lane / 4.
template <int kQ>
__device__ __forceinline__ void load_cols(const uint8_t* src, int64_t ld, int nr, uint32_t lds,
                                          int lane) {
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int row = 16 * q + (lane >> 2);
    const uint8_t* p = src + row * ld + (((lane & 3) ^ col_key(row)) << 4);
    dma16_ptr(row < nr ? p : zero_chunk(), lds + q * 1024);
  }
}

// Sum over this wave's stages s = s0, s0 + ds, .. < ns: load(s, lds) issues a
// stage's loads, of x (the tile's columns, row-staged) and y (kQ tiles of 16 of
// its rows, row- or column-staged).  A slot holds x's, then y's; there are two,
// or three of the smallest.
template <bool kYRows, int kQ, typename Load>
__device__ __forceinline__ void wave_sum(int s0, int ds, int ns, uint32_t base, int lane,
                                         Load&& load, v4f (&acc)[4][4]) {
  constexpr uint32_t kSlotBytes = kOpBytes + kQ * 1024;
  constexpr int kSlots = kWaveBytes / kSlotBytes, kLoads = 4 + kQ;
  static_assert(kSlots == 2 || kSlots == 3);
  const uint32_t fx = base + row_lane(lane);
  const uint32_t fy = base + kOpBytes + (kYRows ? row_lane(lane) : col_lane(lane));
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (s0 + i * ds < ns) load(s0 + i * ds, base + i * kSlotBytes);
  uint32_t slot = 0;
  for (int s = s0; s < ns; s += ds) {
    if (kSlots == 3 && s + 2 * ds < ns) wait_vmcnt<2 * kLoads>();
    else if (s + ds < ns) wait_vmcnt<kLoads>();
    else wait_vmcnt<0>();
    bf16x8 x[4], y[kQ];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = frag_tr<128>((fx + slot) ^ (uint32_t)(i << 5));
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      if constexpr (kYRows) y[i] = frag_tr<128>((fy + slot) ^ (uint32_t)(i << 5));
      else y[i] = lds_load<bf16x8>(fy + slot + i * 1024);
    }
    wait_lgkm0();  // the slot has been read: it may be loaded anew
    sched_fence();
    if (s + kSlots * ds < ns) load(s + kSlots * ds, base + slot);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kQ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[j], acc[i][j], 0, 0, 0);
    slot = slot + kSlotBytes == kSlots * kSlotBytes ? 0 : slot + kSlotBytes;
  }
}

// The eight waves' tiles -> their sum: thread t gets row t / 8, columns
// 8 (t % 8) + 0..7.  16-byte chunks are XOR-swizzled by row.
__device__ __forceinline__ void join_waves(uint32_t lds0, int wid, int lane,
                                           const v4f (&acc)[4][4], float (&out)[8]) {
  const uint32_t own = lds0 + wid * kWaveBytes;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = j * 16 + (lane & 15), c = i * 4 + (lane >> 4);
      lds_store<v4f>(own + row * 256 + ((c ^ (row & 15)) << 4), acc[i][j]);
    }
  __syncthreads();
  const int row = threadIdx.x >> 3, c = (threadIdx.x & 7) * 2;
  v4f lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const uint32_t r = lds0 + w * kWaveBytes + row * 256;
    lo += lds_load<v4f>(r + ((c ^ (row & 15)) << 4));
    hi += lds_load<v4f>(r + (((c + 1) ^ (row & 15)) << 4));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = lo[i], out[4 + i] = hi[i];
}

// Live rows [st, en) of expert e.
__device__ __forceinline__ void expert_rows(const int32_t* psum, int64_t nrows, int align, int e,
                                            int64_t& st, int64_t& en) {
  st = e ? max(0, align_up_i(psum[e - 1], align)) : 0;
  en = min((int64_t)psum[e], nrows);
}

__global__ __launch_bounds__(kThreads) void dgrad_narrow_kernel(
    const uint8_t* __restrict__ dy, const uint8_t* __restrict__ w,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, uint16_t* __restrict__ dx) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * kWaveBytes];
  __shared__ int gp[MOE_MAX_EXPERTS + 1];  // prefix of 64-row groups per expert
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = lds_addr(lds);
  const int64_t nrows = min((int64_t)status[0], capacity);
  if (wid == 0) {
    int sum = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      int ng = 0;
      if (e < E) {
        int64_t st, en;
        expert_rows(psum, nrows, align, e, st, en);
        ng = en > st ? (int)((en - st + T - 1) / T) : 0;
      }
      const int incl = wave_incl_scan_i(ng);
      if (e < E) gp[e] = sum + incl - ng;
      sum += __shfl(incl, 63, 64);
    }
    if (lane == 0) gp[E] = sum;
  }
  __syncthreads();
  const int NT = k / T;
  const uint32_t nitems = (uint32_t)__builtin_amdgcn_readfirstlane(gp[E]) * (uint32_t)NT;
  for (uint32_t base = 0;; base += gridDim.x) {
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
    const int t0 = local / ge * T;
    int64_t st, en;
    expert_rows(psum, nrows, align, e, st, en);
    const int64_t m0 = st + (int64_t)(local % ge) * T;
    const int live = (int)min((int64_t)T, en - m0);
    const uint8_t* a = dy + m0 * n * 2;
    const uint8_t* b = w + ((int64_t)e * n * k + t0) * 2;
    v4f acc[4][4] = {};
    // Only 16-row tiles that hold live rows are loaded and computed (two rows,
    // 5 x 5376 x 576: 12.0 us, 14.7 with all four; 24 rows, 2 x 4224 x 128: 9.2
    // and 12.2).  dy first: the weights first take 4 % longer at 64 rows.
    auto sum = [&](auto q) __attribute__((always_inline)) {
      constexpr int kQ = decltype(q)::value;
      wave_sum<false, kQ>(wid, kWaves, n / kStep, lds0 + wid * kWaveBytes, lane,
                          [&](int s, uint32_t dst) __attribute__((always_inline)) {
                            load_cols<kQ>(a + s * kStep * 2, (int64_t)n * 2, live,
                                          dst + kOpBytes, lane);
                            load_rows(b + (int64_t)s * kStep * k * 2, (int64_t)k * 2, kStep, dst,
                                      lane);
                          },
                          acc);
    };
    if (live <= 16) sum(std::integral_constant<int, 1>());
    else if (live <= 32) sum(std::integral_constant<int, 2>());
    else sum(std::integral_constant<int, 4>());
    float v[8];
    join_waves(lds0, wid, lane, acc, v);
    const int row = threadIdx.x >> 3;
    if (row < live)
      *reinterpret_cast<u32x4*>(dx + (m0 + row) * k + t0 + (threadIdx.x & 7) * 8) = pack8(v);
    __syncthreads();  // the partial tiles have been read
  }
}

template <bool kF32>
__global__ __launch_bounds__(kThreads) void wgrad_narrow_kernel(
    const uint8_t* __restrict__ dy, const uint8_t* __restrict__ x,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, int accumulate, void* __restrict__ dw) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * kWaveBytes];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = lds_addr(lds);
  const int64_t nrows = min((int64_t)status[0], capacity);
  const int NJ = n / T, NT = k / T;
  const int t0 = blockIdx.x % NT * T, j0 = blockIdx.x / NT % NJ * T;
  const int e = blockIdx.x / (NT * NJ);
  int64_t st, en;
  expert_rows(psum, nrows, align, e, st, en);
  const int live = en > st ? (int)(en - st) : 0;
  if (live == 0 && accumulate) return;  // dw[e] stays (uniform)
  const uint8_t* a = dy + (st * n + j0) * 2;
  const uint8_t* b = x + (st * k + t0) * 2;
  v4f acc[4][4] = {};
  wave_sum<true, 4>(wid, kWaves, (live + kStep - 1) / kStep, lds0 + wid * kWaveBytes, lane,
                    [&](int s, uint32_t dst) __attribute__((always_inline)) {
                      const int64_t r = (int64_t)s * kStep;
                      const int nr = (int)min((int64_t)kStep, live - r);
                      load_rows(b + r * k * 2, (int64_t)k * 2, nr, dst, lane);
                      load_rows(a + r * n * 2, (int64_t)n * 2, nr, dst + kOpBytes, lane);
                    },
                    acc);
  float v[8];
  join_waves(lds0, wid, lane, acc, v);
  const int64_t at =
      ((int64_t)e * n + j0 + (threadIdx.x >> 3)) * k + t0 + (threadIdx.x & 7) * 8;
  store_grad8<kF32>(dw, at, v, accumulate);
}

}  // namespace

moe_status launch_dgrad_narrow(const void* dy, const void* w, const int32_t* psum,
                               const int32_t* status, int64_t capacity, int n, int k,
                               int num_experts, int align, void* dx, hipStream_t s) {
  // A workgroup per CU (its LDS): more would only look at the layout and end.
  int64_t grid = ((capacity + T - 1) / T + num_experts) * (int64_t)(k / T);
  if (grid > device_cus()) grid = device_cus();
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL(dgrad_narrow_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s,
                     (const uint8_t*)dy, (const uint8_t*)w, psum, status, capacity, n, k,
                     num_experts, align, (uint16_t*)dx);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

moe_status launch_wgrad_narrow(const void* dy, const void* x, const int32_t* psum,
                               const int32_t* status, int64_t capacity, int n, int k,
                               int num_experts, int align, moe_grad_fmt fmt, int accumulate,
                               void* dw, hipStream_t s) {
  const bool f32 = fmt == MOE_GRAD_F32;
  const int64_t grid = (int64_t)num_experts * (n / T) * (k / T);
  auto kern = f32 ? wgrad_narrow_kernel<true> : wgrad_narrow_kernel<false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0, s, (const uint8_t*)dy,
                     (const uint8_t*)x, psum, status, capacity, n, k, num_experts, align,
                     accumulate, dw);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // namespace moe
