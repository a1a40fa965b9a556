// moe_grouped_dgrad_bf16: input gradient of the grouped bf16 GEMM,
//   dx[m, t] = sum_j dy[m, j] * w[e, j, t] for the live rows m of expert e.
#include "gemm_backward.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;                  // 8 waves, two per SIMD
constexpr int TM = 256, TK = 256;              // output tile: rows x columns of w
constexpr int kStep = 32;                      // reduction per stage of w
constexpr int kRowBytes = TK * 2;              // a staged row of w
constexpr int kWBytes = kStep * kRowBytes;     // 16 KB
constexpr int kWStages = 5;
constexpr int kABytes = TM * 128;              // 32 KB: 64 values of each row of dy (two stages)
constexpr int kAStages = 2;
constexpr int kABase = kWStages * kWBytes;
constexpr int kLds = kABase + kAStages * kABytes;  // 144 KB
constexpr int kLoadWaves = 4;                  // waves 0-3 load w, 4-7 dy
constexpr int kWLoads = 4, kALoads = 8;        // per loading wave and stage (dy: pair of stages)
constexpr int FI = 4, FJ = 8;                  // 16-wide tiles per wave: 64 columns, 128 rows

constexpr int64_t kMinTiles = 80;

// A row of dy is 8 chunks of 16 bytes, XOR-swizzled by row: the 16 rows that
// a fragment reads at one chunk fall on different banks.
__device__ __forceinline__ int a_key(int row) { return (row & 7) ^ ((row >> 3) & 1); }

struct Item {
  int e, t0, live;
  int64_t m0;
};

// The workgroups take the items in rounds.  Where the last round leaves half
// of them idle, its items are cut into their upper and lower 128 rows, which
// waves 0-3 compute in about half the time: PLACEHOLDER.  `whole` items come
// first, then `count - whole` halves.
struct Rounds {
  int64_t whole, count;
  __device__ __forceinline__ Rounds(int64_t items, int64_t grid) {
    const int64_t left = items % grid;
    const bool cut = 2 * left <= grid;
    whole = cut ? items - left : items;
    count = cut ? items + left : items;
  }
};

// Item -> expert, row group and column tile.  Expert e's items are
// [NT * gp[e], NT * gp[e+1]), column-tile-major with the row groups innermost:
// the groups of a tile read the same weights side by side on one XCD.
__device__ __forceinline__ Item decode(int64_t item, int64_t whole, int NT, int E, int align,
                                       int64_t nrows, const int* gp, const int* pe) {
  const int half = item < whole ? -1 : (int)((item - whole) & 1);
  if (half >= 0) item = whole + ((item - whole) >> 1);
  const int q = (int)(item / NT);
  int lo = 0, hi = E - 1;  // last e with gp[e] <= q
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gp[mid] <= q) lo = mid;
    else hi = mid - 1;
  }
  Item it;
  it.e = __builtin_amdgcn_readfirstlane(lo);
  const int g0 = __builtin_amdgcn_readfirstlane(gp[it.e]);
  const int ge = __builtin_amdgcn_readfirstlane(gp[it.e + 1]) - g0;
  const int local = (int)(item - (int64_t)NT * g0);
  it.t0 = local / ge * TK;
  const int st =
      it.e ? max(0, align_up_i(__builtin_amdgcn_readfirstlane(pe[it.e - 1]), align)) : 0;
  it.m0 = st + (int64_t)(local % ge) * TM;
  const int64_t end = min((int64_t)__builtin_amdgcn_readfirstlane(pe[it.e]), nrows);
  it.live = (int)min((int64_t)TM, end - it.m0);
  if (half == 0) it.live = min(it.live, TM / 2);
  if (half == 1) {
    it.m0 += TM / 2;
    it.live = max(it.live - TM / 2, 0);
  }
  return it;
}

// kW: this wave loads w, else dy.
template <bool kW>
__device__ __forceinline__ void run(uint32_t lds0, const int* gp, const int* pe,
                                    const uint8_t* dy, const uint8_t* w, int64_t nrows, int n,
                                    int k, int E, int align, uint16_t* dx, int lane, int wid) {
  const int NT = (k + TK - 1) / TK;
  const Rounds rounds((int64_t)__builtin_amdgcn_readfirstlane(gp[E]) * NT, gridDim.x);
  const int64_t whole = rounds.whole, nitems = rounds.count;
  const int per_xcd = gridDim.x / kXcds;
  const int64_t first = (int64_t)(blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
  const int steps = n / kStep;  // even: n % 128 == 0
  const int wr = wid >> 2, wc = wid & 3;

  // Fragment addresses: w's by transposed reads (see lds_dma.hpp), tile i at
  // piece i ^ key; dy's as rows.
  uint32_t fw, fa;
  {
    const int g = lane >> 4;
    fw = (lds0 + tr_lane_offset(lane) + (wc >> 1) * 256) ^ (uint32_t)((wc & 1) * FI * 32);
    const int row = wr * 128 + (lane & 15);
    fa = lds0 + kABase + (uint32_t)(row * 128 + ((g ^ a_key(row)) << 4));
  }

  // Loading side: this wave's stream of stages, running ahead of the
  // computation across items.
  int64_t d_item = first;
  int d_step = 0, d_live = 0;
  const uint8_t* d_src = nullptr;
  // Load q covers rows r + q * (2 or 8): the offset of row r's chunk (the
  // swizzle repeats with every second load) plus a uniform q * d_pitch.
  uint32_t d_off[2];
  const int64_t d_pitch = kW ? (int64_t)k * 4 : (int64_t)n * 16;
  uint32_t d_slot = 0;
  auto d_open = [&]() __attribute__((always_inline)) {
    d_live = 0;
    if (d_item >= nitems) return;
    const Item it = decode(d_item, whole, NT, E, align, nrows, gp, pe);
    d_live = it.live;
    if constexpr (kW) {
      d_src = w + ((int64_t)it.e * n * k + it.t0) * 2;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = wid * kWLoads * 2 + (lane >> 5);
        const int col = ((lane & 31) ^ (tr_key(row + 2 * j) << 1)) * 8;
        d_off[j] = (uint32_t)(row * k + min(col, k - 8 - it.t0)) * 2u;
      }
    } else {
      d_src = dy + it.m0 * n * 2;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = (wid - kLoadWaves) * kALoads * 8 + (lane >> 3);
        d_off[j] = (uint32_t)(row * n) * 2u + (uint32_t)(((lane & 7) ^ a_key(row + 8 * j)) << 4);
      }
    }
  };
  auto d_load = [&](int q) __attribute__((always_inline)) {
    const uint8_t* p = d_src + q * d_pitch + d_off[q & 1];
    if constexpr (kW) {
      p = d_live > 0 ? p : zero_chunk();
      dma16_ptr(p, lds0 + d_slot + (wid * kWLoads + q) * 1024);
    } else {  // rows that are not live read zeros
      const int row = ((wid - kLoadWaves) * kALoads + q) * 8 + (lane >> 3);
      p = row < d_live ? p : zero_chunk();
      dma16_ptr(p, lds0 + kABase + d_slot + ((wid - kLoadWaves) * kALoads + q) * 1024);
    }
  };
  auto d_advance = [&]() __attribute__((always_inline)) {
    if constexpr (kW) {
      d_slot = d_slot + kWBytes == kWStages * kWBytes ? 0 : d_slot + kWBytes;
      d_src += (int64_t)kStep * k * 2;
      d_step += 1;
    } else {
      d_slot = d_slot + kABytes == kAStages * kABytes ? 0 : d_slot + kABytes;
      d_src += 128;
      d_step += 2;
    }
    if (d_step == steps) {
      d_step = 0;
      d_item += gridDim.x;
      d_open();
    }
  };

  d_open();
#pragma unroll 1
  for (int g = 0; g < (kW ? kWStages : kAStages); ++g) {
#pragma unroll
    for (int q = 0; q < (kW ? kWLoads : kALoads); ++q) d_load(q);
    d_advance();
  }

  uint32_t w_slot = 0, a_slot = 0;  // slots of the stage (pair) to compute
  v4f acc[FI][FJ];
  bf16x8 a[2][FJ], b[2][FI];
  auto read_w = [&](int h, int i, uint32_t slot) __attribute__((always_inline)) {
    b[h][i] = frag_tr<kRowBytes>((fw + slot) ^ (uint32_t)(i << 5));
  };
  auto read_a = [&](int h, int j, uint32_t slot) __attribute__((always_inline)) {
    a[h][j] = lds_load<bf16x8>(((fa + slot) ^ (uint32_t)(h << 6)) + j * 16 * 128);
  };

  for (int64_t item = first; item < nitems; item += gridDim.x) {
    const Item it = decode(item, whole, NT, E, align, nrows, gp, pe);
    const bool busy = wr * 128 < it.live;  // uniform: the wave has live rows
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    wait_vmcnt<0>();
    barrier();
    // Step c (half h of a pair): the next step's stage has landed; the slot of
    // step c (its fragments are in registers) is loaded anew.
    auto half = [&](auto is_busy, auto hh) __attribute__((always_inline)) {
      constexpr bool kBusy = decltype(is_busy)::value;
      constexpr int h = decltype(hh)::value;
      const uint32_t nw = w_slot + kWBytes == kWStages * kWBytes ? 0 : w_slot + kWBytes;
      const uint32_t na = h == 0 ? a_slot : a_slot + kABytes == kAStages * kABytes ? 0
                                                                                : a_slot + kABytes;
      if constexpr (kW) wait_vmcnt<(kWStages - 2) * kWLoads>();
      else if constexpr (h == 1) wait_vmcnt<0>();
      wait_lgkm0();
      barrier();
      sched_fence();
      constexpr int kL = kW ? kWLoads : h == 1 ? kALoads : 0;
#pragma unroll
      for (int u = 0; u < FI * FJ; ++u) {
        if constexpr (kBusy) {
          const int i = u % FI, j = u / FI;
          acc[i][j] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[h][i], a[h][j], acc[i][j], 0, 0, 0);
          sched_fence();
          if (u % 2 == 0 && u / 2 < FI) read_w(h ^ 1, u / 2, nw);
          else if (u % 2 == 0 && u / 2 < FI + FJ) read_a(h ^ 1, u / 2 - FI, na);
        }
        if (u % 2 == 1 && u / 2 < kL) d_load(u / 2);
        sched_fence();
      }
      w_slot = nw;
      a_slot = na;
      if (kL > 0) d_advance();
    };
    if (busy) {
#pragma unroll
      for (int i = 0; i < FI; ++i) read_w(0, i, w_slot);
#pragma unroll
      for (int j = 0; j < FJ; ++j) read_a(0, j, a_slot);
      for (int s = 0; s < steps; s += 2) {
        half(std::true_type(), std::integral_constant<int, 0>());
        half(std::true_type(), std::integral_constant<int, 1>());
      }
      // The lane holds columns t = 4 (lane / 16) + 0..3 of tile i for row
      // lane % 16 of tile j.  Two lane swaps turn the columns of two tiles
      // into 8 neighbouring ones per lane: 16-byte stores, 64 bytes per row.
      const int tc = it.t0 + wc * 64, hf = lane >> 5, r1 = (lane >> 4) & 1;
      if (tc < k) {
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
          const int m = wr * 128 + j * 16 + (lane & 15);
          uint16_t* row = dx + (it.m0 + m) * k + tc + hf * 16 + r1 * 8;
#pragma unroll
          for (int i = 0; i < FI; i += 2) {
            const u32x4 o = pack_tiles(acc[i][j], acc[i + 1][j]);
            if (m < it.live) *reinterpret_cast<u32x4*>(row + i * 16) = o;
          }
        }
      }
    } else {
      for (int s = 0; s < steps; s += 2) {
        half(std::false_type(), std::integral_constant<int, 0>());
        half(std::false_type(), std::integral_constant<int, 1>());
      }
    }
  }
  wait_vmcnt<0>();  // no load may land after the workgroup's LDS has been given away
}

__global__ __launch_bounds__(kThreads, 1) void dgrad_kernel(
    const uint8_t* __restrict__ dy, const uint8_t* __restrict__ w,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, uint16_t* __restrict__ dx) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];  // addresses are XORed
  __shared__ int gp[MOE_MAX_EXPERTS + 1];  // prefix of row groups per expert
  __shared__ int pe[MOE_MAX_EXPERTS];      // end of each expert's live rows
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nrows = min((int64_t)status[0], capacity);
  if (wid == 0) {
    int sum = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      int ng = 0;
      if (e < E) {
        const int64_t st = e ? max(0, align_up_i(psum[e - 1], align)) : 0;
        const int64_t en = min((int64_t)psum[e], nrows);
        ng = en > st ? (int)((en - st + TM - 1) / TM) : 0;
        pe[e] = psum[e];
      }
      const int incl = wave_incl_scan_i(ng);
      if (e < E) gp[e] = sum + incl - ng;
      sum += __shfl(incl, 63, 64);
    }
    if (lane == 0) gp[E] = sum;
  }
  __syncthreads();
  if (wid < kLoadWaves)
    run<true>(lds_addr(lds), gp, pe, dy, w, nrows, n, k, E, align, dx, lane, wid);
  else
    run<false>(lds_addr(lds), gp, pe, dy, w, nrows, n, k, E, align, dx, lane, wid);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_grouped_dgrad_bf16(const void* dy, const void* w, const int32_t* psum,
                                             const int32_t* status, int64_t capacity, int n,
                                             int k, int num_experts, int align, void* dx,
                                             void* stream) {
  const moe_status c = check_backward_sizes(capacity, n, k, num_experts, align);
  if (c != MOE_OK) return c;
  if (!psum || !status || !w) return MOE_ERR_NULL;
  if (capacity > 0 && (!dy || !dx)) return MOE_ERR_NULL;
  if (((uintptr_t)dy % 16) || ((uintptr_t)w % 16) || ((uintptr_t)dx % 16))
    return MOE_ERR_ALIGNMENT;
  if (capacity == 0) return MOE_OK;
  const int64_t max_items = ((capacity + TM - 1) / TM + num_experts) * (int64_t)((k + TK - 1) / TK);
  if (max_items < kMinTiles)
    return launch_dgrad_narrow(dy, w, psum, status, capacity, n, k, num_experts, align, dx,
                               reinterpret_cast<hipStream_t>(stream));
  int64_t grid = device_cus();  // one workgroup per CU, a whole number per XCD
  if (grid > max_items) grid = max_items;
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL(dgrad_kernel, dim3((unsigned)grid), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), (const uint8_t*)dy, (const uint8_t*)w,
                     psum, status, capacity, n, k, num_experts, align, (uint16_t*)dx);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
