// moe_grouped_dgrad_bf16: input gradient of the grouped bf16 GEMM,
//   dx[m, t] = sum_j dy[m, j] * w[e, j, t] for the live rows m of expert e.
//
// Bound by the stream of the weights where experts have few rows (a rank's
// share of about 128 each), by the matrix cores where they have many.
//
//  - One persistent workgroup per CU, tiles of 256 rows x 256 columns, eight
//    waves (two per SIMD) of 128 rows x 64 columns, v_mfma_f32_16x16x32_bf16
//    with w as the first operand, so that a lane ends up with neighbouring
//    columns of a row.  128 x 128 tiles (waves of 64 x 32) where the larger
//    ones leave CUs idle, 64 x 64 (grad_narrow.hip) where those do.
//  - The sum runs over w's rows, so w is staged as rows and read through
//    ds_read_b64_tr_b16 (lds_dma.hpp); dy's rows hold the sum's axis and are
//    read as they are.
//  - Operands go HBM -> LDS directly: waves 0-3 load w (32 rows a stage, five
//    stages, four steps ahead), waves 4-7 dy (64 columns of 256 rows, whole
//    128-byte lines, two stages).  The load counter is per wave, so each
//    stream keeps its own depth (128 x 128: four stages of dy).  Both run ahead
//    across tiles.  Rows that are not live are loaded from a chunk of zeros
//    and cost no traffic; a wave whose rows hold none skips its MFMAs.
//  - What it reaches: 105 us at one rank's share (1024 rows, 8 x 4096 x 7168:
//    4.7 TB/s), 418 us at 18432 uneven rows of 6144 x 2048 (1.11 PFLOP/s) and
//    806 at 4096 x 6144 (1.15; with zeros as inputs 649: power, as in
//    wgrad.hip).
#include "gemm_backward.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;                  // 8 waves, two per SIMD
constexpr int kStep = 32;                      // reduction per step
constexpr int kWBytes = 16384;                 // a stage of w: 32 x 256 or 64 x 128 values
constexpr int kWStages = 5;
constexpr int kARing = 65536;                  // dy: 64 values (two steps) of a tile's rows a stage
constexpr int kABase = kWStages * kWBytes;
constexpr int kLds = kABase + kARing;          // 144 KB
constexpr int kLoadWaves = 4;                  // waves 0-3 load w, 4-7 dy
constexpr int kWLoads = 4;                     // per loading wave and stage
// Few rows leave little to compute while the loads are under way: the smaller
// tiles have four stages of dy instead of two.
template <int TK>
struct Shape {
  static constexpr int kRows = TK;
  static constexpr int kABytes = kRows * 128;         // a stage of dy
  static constexpr int kAStages = kARing / kABytes;   // 2 or 4
  static constexpr int kALoads = kRows / 32;          // per loading wave and stage
  static constexpr int FI = TK / 64, FJ = kRows / 32;  // 16-wide tiles per wave: columns, rows
};

// Square tiles of t rows and columns to expect.  The rows of an expert are only
// known on the device: as many live ones as fit the capacity with the worst
// alignment, evenly spread, half a tile lost by each expert.
inline int64_t expected_tiles(int64_t capacity, int k, int num_experts, int align, int t) {
  const int64_t experts = min((int64_t)num_experts, capacity / align);  // with rows
  const int64_t live = capacity - experts * (align - 1);
  return max(experts, live / t + experts / 2) * ((k + t - 1) / t);
}
// Which kernel: the smallest tiles that the CUs hold at once, since each step of
// a tile takes its loads' latency or longer.  Measured with 64 / 128 / 256, rows
// per expert: 64 rows, 8 x 2048 x 1024, 13 / 19 / 32 us; 256 rows there, 27 / 21 /
// 32; 512 rows, 2 x 7168 x 2048, 74 / 53 / 94; 8 rows, 8 x 4096 x 2048, 26 / 28 /
// 59; more than one round of 128 x 128 tiles: 512 rows, 8 x 2048 x 1024, 43 / 36 /
// 33; 128 rows, 8 x 4096 x 7168, 179 / 128 / 104.
// A capacity far above the live rows (a layer class allocates topk rows for every
// row received, of which an expert-parallel rank uses few) makes the rule expect
// tiles that are not there, and take larger ones than the live rows want: 1024
// rows, 8 x 2048 x 1024, 19.5 us in a buffer of 1920 rows, 32 in one of 33664; 8 x
// 7168 x 2048, 81 and 121; 8 x 4096 x 7168, 106 in both.
constexpr int64_t kFull = 256;

// A row of dy is 8 chunks of 16 bytes, XOR-swizzled by row so that the 16
// lanes that a 16-byte LDS read serves at once fall on different banks, whether
// they are 16 consecutive ones or, as counted, lanes 0-3 and 12-15 of one row
// group with 4-11 of the next (the key (row & 7) ^ (row >> 3 & 1), which only
// looks at the former, lost 40% of the LDS cycles to conflicts).
__device__ __forceinline__ int a_key(int row) { return (row >> 1) & 7; }

struct Item {
  int e, t0, live;
  int64_t m0;
};

// The workgroups take the items in rounds.  Where the last round leaves half
// of them idle, its items (256 x 256 ones) are cut into their upper and lower 128 rows, which
// waves 0-3 compute in about half the time (18432 rows, 6144 x 2048: 454 ->
// 420 us; 16384 rows, 2 x 2048 x 1024: 97 -> 83).  `whole` items come
// first, then `count - whole` halves.
// Items fit 32 bits: at most 2^22 + 2^10 row groups of 2^7 column tiles, twice that
// many halves (256 x 256); 2^23 + 2^10 groups of 2^8 (128 x 128).
struct Rounds {
  uint32_t whole, count;
  __device__ __forceinline__ Rounds(uint32_t items, uint32_t grid, bool halves) {
    const uint32_t left = items % grid;
    const bool cut = 2 * left <= grid && halves;
    whole = cut ? items - left : items;
    count = cut ? items + left : items;
  }
};

// Item -> expert, row group and column tile.  Expert e's items are
// [NT * gp[e], NT * gp[e+1]), column-tile-major with the row groups innermost:
// the groups of a tile read the same weights side by side on one XCD.
template <int TK>
__device__ __forceinline__ Item decode(uint32_t item, uint32_t whole, int NT, int E, int align,
                                       int64_t nrows, const int* gp, const int* pe) {
  const int half = item < whole ? -1 : (int)((item - whole) & 1);
  if (half >= 0) item = whole + ((item - whole) >> 1);
  const int q = (int)(item / (uint32_t)NT);
  int lo = 0, hi = E - 1;  // last e with gp[e] <= q
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gp[mid] <= q) lo = mid;
    else hi = mid - 1;
  }
  constexpr int TM = Shape<TK>::kRows;
  Item it;
  it.e = __builtin_amdgcn_readfirstlane(lo);
  const int g0 = __builtin_amdgcn_readfirstlane(gp[it.e]);
  const int ge = __builtin_amdgcn_readfirstlane(gp[it.e + 1]) - g0;
  const int local = (int)(item - (uint32_t)NT * (uint32_t)g0);
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

// TK: columns of an output tile, 256 or 128.  kW: this wave loads w, else dy.
template <int TK, bool kW>
__device__ __forceinline__ void run(uint32_t lds0, const int* gp, const int* pe,
                                    const uint8_t* dy, const uint8_t* w, int64_t nrows, int n,
                                    int k, int E, int align, uint16_t* dx, int lane, int wid) {
  constexpr int kRowBytes = TK * 2;                      // a staged row of w
  constexpr int kStageRows = kWBytes / kRowBytes;        // 32 or 64
  constexpr int kStageSteps = kStageRows / kStep;        // steps per stage of w: 1 or 2
  constexpr int kLoadRows = 1024 / kRowBytes;            // rows of w per load: 2 or 4
  using S = Shape<TK>;
  constexpr int FI = S::FI, FJ = S::FJ, kALoads = S::kALoads;
  constexpr int kWaveRows = S::kRows / 2;
  const int NT = (k + TK - 1) / TK;
  const Rounds rounds((uint32_t)__builtin_amdgcn_readfirstlane(gp[E]) * NT, gridDim.x,
                      TK == 256);
  const uint32_t whole = rounds.whole, nitems = rounds.count;
  const int steps = n / kStep;  // even: n % 128 == 0
  const int wr = wid >> 2, wc = wid & 3;

  // Fragment addresses: w's by transposed reads (see lds_dma.hpp), tile i at
  // piece i ^ key; dy's as rows.
  uint32_t fw, fa;
  {
    const int g = lane >> 4;
    const int piece = wc * FI;  // 32-byte pieces, eight to 256 bytes
    fw = (lds0 + tr_lane_offset<kRowBytes>(lane) + (piece >> 3) * 256) ^
         (uint32_t)((piece & 7) << 5);
    const int row = wr * kWaveRows + (lane & 15);
    fa = lds0 + kABase + (uint32_t)(row * 128 + ((g ^ a_key(row)) << 4));
  }

  // Loading side: this wave's stream of stages, running ahead of the
  // computation across items.
  uint32_t d_base = 0;  // the round
  int d_step = 0, d_live = 0;
  const uint8_t* d_src = nullptr;
  // Load q covers rows r + q * (kLoadRows or 8): the offset of row r's chunk
  // (one of two, by the swizzle) plus a uniform q * d_pitch.
  uint32_t d_off[2] = {};
  const int64_t d_pitch = kW ? (int64_t)k * 2 * kLoadRows : (int64_t)n * 16;
  uint32_t d_slot = 0;
  auto d_open = [&]() __attribute__((always_inline)) {
    d_live = 0;
    const uint32_t d_item = round_item(d_base, nitems);
    if (d_item >= nitems) return;
    const Item it = decode<TK>(d_item, whole, NT, E, align, nrows, gp, pe);
    d_live = it.live;
    if constexpr (kW) {
      d_src = w + ((int64_t)it.e * n * k + it.t0) * 2;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        constexpr int kLanes = 64 / kLoadRows;  // per row
        const int row = wid * kWLoads * kLoadRows + lane / kLanes;
        const int col = (lane % kLanes ^ (tr_key(row + (TK == 256 ? 2 : 8) * j) << 1)) * 8;
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
    const uint8_t* p = d_src + q * d_pitch + d_off[kW && TK == 128 ? q >> 1 : q & 1];
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
      d_src += (int64_t)kStageRows * k * 2;
      d_step += kStageSteps;
    } else {
      d_slot = d_slot + S::kABytes == kARing ? 0 : d_slot + S::kABytes;
      d_src += 128;
      d_step += 2;
    }
    if (d_step == steps) {
      d_step = 0;
      d_base += gridDim.x;
      d_open();
    }
  };

  d_open();
#pragma unroll 1
  for (int g = 0; g < (kW ? kWStages : S::kAStages); ++g) {
#pragma unroll
    for (int q = 0; q < (kW ? kWLoads : kALoads); ++q) d_load(q);
    d_advance();
  }

  uint32_t w_slot = 0, a_slot = 0;  // slots of the stage (pair) to compute
  v4f acc[FI][FJ];
  bf16x8 a[2][FJ], b[2][FI];
  auto read_w = [&](int h, int i, uint32_t slot) __attribute__((always_inline)) {
    const int row = kStageSteps == 2 ? h * kStep : 0;
    b[h][i] = frag_tr<kRowBytes>(((fw + slot) ^ (uint32_t)(i << 5)) + row * kRowBytes);
  };
  auto read_a = [&](int h, int j, uint32_t slot) __attribute__((always_inline)) {
    a[h][j] = lds_load<bf16x8>(((fa + slot) ^ (uint32_t)(h << 6)) + j * 16 * 128);
  };

  for (uint32_t base = 0;; base += gridDim.x) {
    const uint32_t item = round_item(base, nitems);
    if (item >= nitems) break;
    const Item it = decode<TK>(item, whole, NT, E, align, nrows, gp, pe);
    const bool busy = wr * kWaveRows < it.live;  // uniform: the wave has live rows
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    wait_vmcnt<0>();
    barrier();
    // One step (half h of a pair).  Where the next step starts a new stage: it
    // has landed, and the slot that this step's fragments came from (they are
    // in registers) is loaded anew.
    auto half = [&](auto is_busy, auto hh) __attribute__((always_inline)) {
      constexpr bool kBusy = decltype(is_busy)::value;
      constexpr int h = decltype(hh)::value;
      constexpr bool kNewW = kStageSteps == 1 || h == 1, kNewA = h == 1;
      const uint32_t nw = !kNewW ? w_slot : w_slot + kWBytes == kWStages * kWBytes
                                                ? 0
                                                : w_slot + kWBytes;
      const uint32_t na = !kNewA ? a_slot : a_slot + S::kABytes == kARing ? 0 : a_slot + S::kABytes;
      if constexpr (kNewW) {
        if constexpr (kW) wait_vmcnt<(kWStages - 2) * kWLoads>();
        else if (kNewA) wait_vmcnt<(S::kAStages - 2) * kALoads>();
        wait_lgkm0();
        barrier();
      }
      sched_fence();
      constexpr int kL = kW ? (kNewW ? kWLoads : 0) : kNewA ? kALoads : 0;
#pragma unroll
      for (int u = 0; u < FI * FJ; ++u) {
        if constexpr (kBusy) {
          const int i = u % FI, j = u / FI;
          acc[i][j] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[h][i], a[h][j], acc[i][j], 0, 0, 0);
          sched_fence();
          if (TK == 128 && u < FI + FJ) {  // 8 MFMAs: a read beside all but two
            if (u < FI) read_w(h ^ 1, u, nw);
            else read_a(h ^ 1, u - FI, na);
          } else if (TK == 256 && u % 2 == 0 && u / 2 < FI + FJ) {
            if (u / 2 < FI) read_w(h ^ 1, u / 2, nw);
            else read_a(h ^ 1, u / 2 - FI, na);
          }
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
      const int tc = it.t0 + wc * FI * 16, hf = lane >> 5, r1 = (lane >> 4) & 1;
      if (tc < k) {
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
          const int m = wr * kWaveRows + j * 16 + (lane & 15);
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

template <int TK>
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
    constexpr int TM = Shape<TK>::kRows;
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
    run<TK, true>(lds_addr(lds), gp, pe, dy, w, nrows, n, k, E, align, dx, lane, wid);
  else
    run<TK, false>(lds_addr(lds), gp, pe, dy, w, nrows, n, k, E, align, dx, lane, wid);
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
  const int64_t out = capacity * k * 2;
  if (overlap(dx, out, dy, capacity * n * 2) ||
      overlap(dx, out, w, (int64_t)num_experts * n * k * 2))
    return MOE_ERR_UNSUPPORTED;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (expected_tiles(capacity, k, num_experts, align, kNarrowTile) <= kFull)
    return launch_dgrad_narrow(dy, w, psum, status, capacity, n, k, num_experts, align, dx, st);
  const bool half_wide = expected_tiles(capacity, k, num_experts, align, 128) <= kFull;
  int64_t grid = device_cus();  // one workgroup per CU, a whole number per XCD
  const int t = half_wide ? 128 : 256;
  const int64_t most = 2 * ((capacity + t - 1) / t + num_experts) * ((k + t - 1) / t);  // halves
  if (grid > most) grid = most;
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  auto kern = half_wide ? dgrad_kernel<128> : dgrad_kernel<256>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0, st, (const uint8_t*)dy,
                     (const uint8_t*)w, psum, status, capacity, n, k, num_experts, align,
                     (uint16_t*)dx);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
