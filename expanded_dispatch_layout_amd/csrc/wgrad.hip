// moe_grouped_wgrad_bf16: weight gradient of the grouped bf16 GEMM,
//   dw[e, j, t] = sum over the live rows m of expert e of dy[m, j] * x[m, t].
//
// Bound by the matrix cores for long experts (256 x 256 tiles: 128 flop per
// byte read into LDS), by the write of dw for short ones (a rank's share of
// about 128 rows an expert does 128 flop for each 2 or 4 bytes of dw).
//
//  - One persistent workgroup per CU, 256 x 256 outputs, eight waves (two per
//    SIMD) of 64 dy columns x 128 x columns: 8 x 4 v_mfma_f32_16x16x32_bf16
//    per 32 rows.  128 x 128 outputs (waves of 32 x 64, a ring of eight stages)
//    where those leave CUs idle, 64 x 64 where these do.  (Measured at 18432
//    rows, 4096 x 6144: four waves of 128 x 128 are bound by issue, 850 us
//    against 808 then; 32x32x16 MFMAs draw more power, 879.)
//  - The sum runs over the rows, along which neither operand is contiguous:
//    both are staged as rows (coalesced loads) and read through
//    ds_read_b64_tr_b16 (lds_dma.hpp).
//  - Stages of 32 rows of both operands, HBM -> LDS directly, in a ring of
//    five, loaded three to four steps ahead and across tiles: the next tile's
//    first stages arrive during this one's epilogue.  Rows past an expert's
//    last live one are loaded from a chunk of zeros, so alignment pads never
//    enter a product, whatever they hold.
//  - Fragments are double-buffered in registers: a step's 32 MFMAs run while
//    the next one's 24 reads are under way, with one barrier per step.
//  - What it reaches: 766 us at 18432 rows of 4096 x 6144 (1.21 PFLOP/s; the
//    library's plain product of that layout and size takes 890); at one rank's
//    share (1024 rows, 8 x 4096 x 7168) 116 us writing bf16 and 211 adding to it,
//    189 and 381 in fp32 (4.2 to 5.1 TB/s).  The large one is bound by power: with zeros as inputs
//    the same instructions take 612 us.
#include <math.h>

#include <type_traits>

#include "gemm_backward.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int kStep = 32;         // rows per stage
constexpr int kLds = 160 * 1024;  // all of the CU's

// Output tiles are T x T, 256 or 128.
template <int T>
struct Shape {
  static constexpr int kRowBytes = T * 2;
  static constexpr int kOpBytes = kStep * kRowBytes;  // one operand of a stage
  static constexpr int kStageBytes = 2 * kOpBytes;    // 32 or 16 KB
  static constexpr int kStages = T == 256 ? 5 : 8;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kLoads = T / 64;               // DMA instructions per wave and stage
  static constexpr int FI = T / 32, FJ = T / 64;      // 16-wide tiles per wave: x, dy columns
};

constexpr int64_t kFullTiles = 256;  // one per CU

struct Tile {
  int e, j0, t0, z;  // expert, first dy and x column, part of the sum
  int64_t st;        // first row
  int live;          // rows
  bool idle;         // the expert has none at all
};

// Stages of a tile: computed in pairs, so an odd count gets one of zeros.
__device__ __forceinline__ int stages_of(int live) {
  return 2 * ((live + 2 * kStep - 1) / (2 * kStep));
}

// Items of one expert: panels of 8 tiles along t, j-major inside a panel, so
// that the 32 neighbouring items of an XCD's CUs are a 4 x 8 block and share
// their operands in its L2.
template <int T>
__device__ __forceinline__ Tile decode(uint32_t item, int NJ, int NT, int splits,
                                       const int32_t* psum, int64_t nrows, int align) {
  Tile t;
  const uint32_t per = NJ * NT;
  t.z = splits > 1 ? (int)(item % (uint32_t)splits) : 0;
  if (splits > 1) item /= (uint32_t)splits;
  t.e = (int)(item / per);
  const int local = (int)(item - t.e * per);
  const int panel = local / (8 * NJ);
  const int rem = local - panel * 8 * NJ;
  const int w = min(8, NT - panel * 8);
  t.j0 = rem / w * T;
  t.t0 = (panel * 8 + rem % w) * T;
  t.st = t.e ? max(0, align_up_i(psum[t.e - 1], align)) : 0;
  const int64_t en = min((int64_t)psum[t.e], nrows);
  t.live = en > t.st ? (int)(en - t.st) : 0;
  t.idle = t.live == 0;
  if (splits > 1) {  // part z: an even share of the stages, in pairs
    const int share = 2 * ((stages_of(t.live) / 2 + splits - 1) / splits) * kStep;
    t.st += (int64_t)t.z * share;
    t.live = max(0, min(share, t.live - t.z * share));
  }
  return t;
}

// kF32: dw is fp32, else bf16.  kAdd: the sums are added to it.  kParts: part z
// of a split sum goes to dw[z][E][n][k].
template <int T, bool kF32, bool kAdd, bool kParts>
__global__ __launch_bounds__(kThreads, 1) void wgrad_kernel(
    const uint8_t* __restrict__ dy, const uint8_t* __restrict__ x,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, int splits, void* __restrict__ dw) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];  // addresses are XORed
  using S = Shape<T>;
  constexpr int kRowBytes = S::kRowBytes, kOpBytes = S::kOpBytes, kStageBytes = S::kStageBytes;
  constexpr int kStages = S::kStages, kRing = S::kRing, kLoads = S::kLoads;
  constexpr int FI = S::FI, FJ = S::FJ;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = lds_addr(lds);
  const int64_t nrows = min((int64_t)status[0], capacity);
  const int NJ = (n + T - 1) / T, NT = (k + T - 1) / T;
  // At most 2^24 tiles (1024 experts, 128 x 128), and a split sum has few.
  const uint32_t nitems = (uint32_t)E * NJ * NT * splits;

  // The first round behind that at `base` that may have an item whose expert
  // has rows, expert e having none: 64 experts are looked at at once, since each
  // look is a round trip to memory (8 of 256 experts with a row, 4096 x 7168,
  // adding to bf16: 213 us, against 381 tile by tile and 202 for those 8 experts
  // alone).  Only where dw is added to: elsewhere every tile of such an expert
  // is written, at the memory's rate (256 experts: 2.7 ms for 15 GB).
  auto skip_idle = [&](uint32_t base, int e) __attribute__((always_inline)) -> uint32_t {
    for (int q0 = e + 1; q0 < E; q0 += 64) {
      const int q = q0 + lane;
      bool live = false;
      if (q < E)
        live = min((int64_t)psum[q], nrows) > (int64_t)max(0, align_up_i(psum[q - 1], align));
      const uint64_t mask = __ballot(live);
      if (mask) {
        const uint32_t at =
            (uint32_t)(q0 + __builtin_ctzll(mask)) * (uint32_t)(NJ * NT) * (uint32_t)splits;
        return max(base + gridDim.x, at / gridDim.x * gridDim.x);
      }
    }
    return nitems;
  };

  // Fragment addresses within a stage: tile i of a wave is its 32-byte piece
  // i ^ key of a row, so one lane base serves all of them through an XOR.
  const int wj = wid >> 1, wt = wid & 1;
  uint32_t fx, fy;  // x, dy
  {
    const uint32_t base = lds0 + tr_lane_offset<kRowBytes>(lane);
    const int px = wt * FI, py = wj * FJ;  // 32-byte pieces, eight to 256 bytes
    fx = (base + kOpBytes + (px >> 3) * 256) ^ (uint32_t)((px & 7) << 5);
    fy = (base + (py >> 3) * 256) ^ (uint32_t)((py & 7) << 5);
  }

  // DMA side: the next stage to load.
  uint32_t d_base = 0;  // the round
  int d_left = 0;    // rows left of its tile (<= 0: a stage of zeros)
  int d_stages = 0;  // stages left of its tile
  const uint8_t *d_dy = nullptr, *d_x = nullptr;
  constexpr int kHalf = kLoads / 2;            // of each operand: 2 or 1
  constexpr int kLoadRows = 1024 / kRowBytes;  // 2 or 4
  constexpr int kLanes = 64 / kLoadRows;       // per row
  uint32_t d_offa[kHalf] = {}, d_offb[kHalf] = {};  // x, dy: offsets of this lane's chunks
  uint32_t d_slot = 0;            // LDS offset of the next slot
  auto d_open = [&]() __attribute__((always_inline)) {  // next tile that has rows
    while (true) {
      const uint32_t d_item = round_item(d_base, nitems);
      if (d_item >= nitems) break;
      const Tile t = decode<T>(d_item, NJ, NT, splits, psum, nrows, align);
      if (t.live > 0) {
        d_left = t.live;
        d_stages = stages_of(t.live);
        d_dy = dy + (t.st * n + t.j0) * 2;
        d_x = x + (t.st * k + t.t0) * 2;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          const int row = wid * 4 + j * kLoadRows + lane / kLanes;
          const int col = ((lane % kLanes) ^ (tr_key(row) << 1)) * 8;
          d_offb[j] = (uint32_t)(row * n + min(col, n - 8 - t.j0)) * 2u;
          d_offa[j] = (uint32_t)(row * k + min(col, k - 8 - t.t0)) * 2u;
        }
        return;
      }
      d_base = kAdd && t.idle ? skip_idle(d_base, t.e) : d_base + gridDim.x;
    }
  };
  // Load q of the next stage: dy rows first, then x.  Rows past the
  // tile's last live one, and every row once there is no tile left, read
  // zeros, so that each step issues the same loads without a branch.
  const int d_row = wid * 4 + lane / kLanes;  // this lane's row in load 0
  auto d_load = [&](int q) __attribute__((always_inline)) {
    const int j = q % kHalf;
    const uint8_t* p = q < kHalf ? d_dy + d_offb[j] : d_x + d_offa[j];
    p = d_row + kLoadRows * j < d_left ? p : zero_chunk();
    dma16_ptr(p, lds0 + d_slot + (wid * kHalf + j) * 1024 + (q < kHalf ? 0 : kOpBytes));
  };
  auto d_advance = [&]() __attribute__((always_inline)) {
    d_slot = d_slot + kStageBytes == kRing ? 0 : d_slot + kStageBytes;
    d_left -= kStep;
    d_dy += (int64_t)kStep * n * 2;
    d_x += (int64_t)kStep * k * 2;
    if (--d_stages <= 0 && d_base < nitems) {
      d_base += gridDim.x;
      d_open();
    }
  };

  d_open();
  for (int g = 0; g < kStages - 1; ++g) {
    for (int q = 0; q < kLoads; ++q) d_load(q);
    d_advance();
  }

  uint32_t c_slot = 0;  // slot of the stage to compute
  v4f acc[FI][FJ];
  bf16x8 a[2][FI], b[2][FJ];

  for (uint32_t base = 0, next;; base = next) {
    const uint32_t item = round_item(base, nitems);
    if (item >= nitems) break;
    const Tile t = decode<T>(item, NJ, NT, splits, psum, nrows, align);
    const int steps = stages_of(t.live);
    next = kAdd && t.idle ? skip_idle(base, t.e) : base + gridDim.x;
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    if (steps > 0) {
      wait_vmcnt<0>();
      barrier();
#pragma unroll
      for (int j = 0; j < FJ; ++j) b[0][j] = frag_tr<kRowBytes>((fy + c_slot) ^ (j << 5));
#pragma unroll
      for (int i = 0; i < FI; ++i) a[0][i] = frag_tr<kRowBytes>((fx + c_slot) ^ (i << 5));
      for (int s = 0; s < steps; s += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t nslot = c_slot + kStageBytes == kRing ? 0 : c_slot + kStageBytes;
          const uint32_t nx = fx + nslot, ny = fy + nslot;
          wait_vmcnt<(kStages - 3) * kLoads>();
          barrier();
          sched_fence();
#pragma unroll
          for (int u = 0; u < FI * FJ; ++u) {
            const int i = u / FJ, j = u % FJ;
            acc[i][j] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[h][i], b[h][j], acc[i][j], 0, 0, 0);
            sched_fence();
            if (T == 128) {  // 8 MFMAs: a read or a load beside each
              if (u < FJ) b[h ^ 1][u] = frag_tr<kRowBytes>(ny ^ (u << 5));
              else if (u < FJ + FI) a[h ^ 1][u - FJ] = frag_tr<kRowBytes>(nx ^ ((u - FJ) << 5));
              else d_load(u - FJ - FI);
            } else if (u % 2 == 0 && u / 2 < FJ)
              b[h ^ 1][u / 2] = frag_tr<kRowBytes>(ny ^ ((u / 2) << 5));
            else if (u % 2 == 0 && u / 2 < FJ + FI)
              a[h ^ 1][u / 2 - FJ] = frag_tr<kRowBytes>(nx ^ ((u / 2 - FJ) << 5));
            else if (u % 4 == 1 && u / 4 < kLoads) d_load(u / 4);
            sched_fence();
          }
          c_slot = nslot;
          d_advance();
        }
      }
    } else if (kAdd) {
      continue;  // dw[e] stays
    }
    // Epilogue.  The lane holds columns t = 4 (lane / 16) + 0..3 of tile i for
    // row j = lane % 16 of tile j.  Each wave passes 16 rows at a time through
    // its 4 KB of the slot that the last stage has left (16-byte chunks
    // XOR-swizzled by row), so that a store covers 256 bytes of 4 rows instead
    // of 64 bytes of 16 (one rank's share, 1024 rows of 8 x 4096 x 7168, through
    // the caches: 137 us against 160 in bf16, 394 against 432 accumulating in
    // fp32).
    if constexpr (T == 256) barrier();  // every wave has read that slot
    const uint32_t own = lds0 + (uint32_t)wid * 4096u +
                         (T == 256 ? (c_slot == 0 ? kRing : c_slot) - kStageBytes : kRing);
    const int jc = t.j0 + wj * FJ * 16, tc = t.t0 + wt * FI * 16;
    const int fr = lane & 15, g = lane >> 4;
    // 64 columns (tiles i0..) of 16 rows into LDS as fp32.
    auto stage = [&](int i0, int j) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lds_store<v4f>(own + fr * 256 + (((i * 4 + g) ^ fr) << 4), acc[i0 + i][j]);
    };
    auto staged = [&](int r, int c) __attribute__((always_inline)) {  // row r, chunk c
      return lds_load<v4f>(own + r * 256 + ((c ^ r) << 4));
    };
    // dw is not read again here: its accesses pass the caches by (one rank's
    // share: 114 us against 137 in bf16, 378 against 394 accumulating in fp32;
    // a backward pass and AdamW around them 2-3% less).  The parts of a split
    // sum are read next by the join and stay in them.
    if (jc < n) {
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int64_t row0 = ((int64_t)t.z * E + t.e) * n + jc + j * 16;
        if constexpr (kF32) {
#pragma unroll
          for (int i0 = 0; i0 < FI; i0 += 4) {
            if (tc + i0 * 16 >= k) break;  // k is a multiple of 64
            float* o = (float*)dw + (row0 + g) * k + tc + i0 * 16 + fr * 4;  // rows 4 q + g
            v4f old[4];
            if constexpr (kAdd) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                old[q] = __builtin_nontemporal_load(
                    reinterpret_cast<const v4f*>(o + 4 * q * (int64_t)k));
            }
            stage(i0, j);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v4f v = staged(4 * q + g, fr);
              if constexpr (kAdd) v += old[q];
              v4f* to = reinterpret_cast<v4f*>(o + 4 * q * (int64_t)k);
              if constexpr (kParts) *to = v;
              else __builtin_nontemporal_store(v, to);
            }
          }
        } else if constexpr (kAdd) {  // bf16 sums are added in fp32
#pragma unroll
          for (int i0 = 0; i0 < FI; i0 += 4) {
            if (tc + i0 * 16 >= k) break;
            const int r = lane >> 3, c = (lane & 7) * 2;  // rows 8 q + r
            uint16_t* o = (uint16_t*)dw + (row0 + r) * k + tc + i0 * 16 + c * 4;
            u32x4 old[2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
              old[q] = __builtin_nontemporal_load(
                  reinterpret_cast<const u32x4*>(o + 8 * q * (int64_t)k));
            stage(i0, j);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const v4f x = staged(8 * q + r, c), y = staged(8 * q + r, c + 1);
              float v[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const u32x4 b = old[q];
                v[e] = x[e] + __uint_as_float(e & 1 ? b[e / 2] & 0xffff0000u : b[e / 2] << 16);
                v[4 + e] =
                    y[e] + __uint_as_float(e & 1 ? b[2 + e / 2] & 0xffff0000u : b[2 + e / 2] << 16);
              }
              __builtin_nontemporal_store(pack8(v),
                                          reinterpret_cast<u32x4*>(o + 8 * q * (int64_t)k));
            }
          }
        } else {  // all columns as bf16, kC chunks a row
          constexpr int kC = 2 * FI, kPass = 64 / kC;
#pragma unroll
          for (int i = 0; i < FI; ++i) {
            typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
            lds_store<u32x2>(
                own + fr * kC * 16 + (((2 * i + (g >> 1)) ^ (fr % kC)) << 4) + (g & 1) * 8,
                u32x2{pk_bf16(acc[i][j][0], acc[i][j][1]), pk_bf16(acc[i][j][2], acc[i][j][3])});
          }
#pragma unroll
          for (int q = 0; q < 16 / kPass; ++q) {
            const int r = q * kPass + lane / kC, c = lane % kC;
            const u32x4 v = lds_load<u32x4>(own + r * kC * 16 + ((c ^ (r % kC)) << 4));
            if (tc + c * 8 < k)
              __builtin_nontemporal_store(
                  v, reinterpret_cast<u32x4*>((uint16_t*)dw + (row0 + r) * k + tc + c * 8));
          }
        }
      }
    }
  }
  wait_vmcnt<0>();  // no load may land after the workgroup's LDS has been given away
}

// dw = (dw +) the sum of the parts, in their order.  One wave per workgroup and
// several parts' loads in flight: the sum over many parts of a small dw is
// bound by latency.
constexpr int kJoinThreads = 64;
template <bool kF32>
__global__ __launch_bounds__(kJoinThreads) void wgrad_join_kernel(const float* __restrict__ part,
                                                         int splits, int64_t count,
                                                         int accumulate, void* __restrict__ dw) {
  const int64_t at = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 8;
  if (at >= count) return;
  v4f lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll 8
  for (int z = 0; z < splits; ++z) {
    const v4f* p = reinterpret_cast<const v4f*>(part + z * count + at);
    lo += p[0];
    hi += p[1];
  }
  const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  store_grad8<kF32>(dw, at, v, accumulate);
}

}  // namespace
}  // namespace moe

using namespace moe;

namespace moe {
namespace {

int64_t tiles_of(int n, int k, int num_experts, int t) {
  return (int64_t)num_experts * ((n + t - 1) / t) * ((k + t - 1) / t);
}

// Which tiles: the smallest that the CUs hold at once, since a step of a tile
// takes its loads' latency or longer.  With long sums the 256 x 256 ones, split
// over workgroups (wgrad_splits).  Measured with 64 (grad_narrow.hip) / 128 /
// 256, rows per expert: 1024 x 1024, one expert (256 tiles of 64), 16 rows 4.0 /
// 5.5 / 7.4 us, 1024 rows 8.4 / 14.4 / 19.9, 4096 rows 20 / 42 / 29, 8192 rows 36 /
// 78 / 38; 1024 x 1024, four (256 tiles of 128), 16 rows 11.9 / 6.5 / 8.3, 512 rows
// 20 / 11 / 17, 2048 rows 40 / 26 / 38, 4096 rows 70 / 46 / 50; 4096 x 1024, one,
// 8192 rows 137 / 85 / 78.
// Two rounds of 128 take as long as one of 256 where experts are even, and less
// where they are not, since fewer CUs wait for the longest: 1024 x 1024, eight,
// 4096 rows even 17.9 / 18.4 us, 6400 rows of which 43 % are one expert's 40 / 62;
// three rounds lose more (384 x 1728, fourteen, 5473 rows even 21.2 / 16.3).
// The border in rows serves both; between it and about 8192 rows of one expert 64
// would still be a little ahead.  Rows are those of a full buffer: see
// wgrad_splits.
constexpr int64_t kShortRows = 4608;
int tile_of(int64_t capacity, int n, int k, int num_experts) {
  const int64_t rows = capacity / num_experts;
  if (tiles_of(n, k, num_experts, 64) <= kFullTiles && rows <= kShortRows) return 64;
  const int64_t rounds = (tiles_of(n, k, num_experts, 128) + kFullTiles - 1) / kFullTiles;
  if (rounds <= 2 && rounds * rows <= kShortRows) return 128;
  return 256;
}

// Parts that each expert's sum is cut into where the tiles leave CUs idle.  A
// stage of a tile takes about 0.5 us, so the sum of an average expert's R rows
// takes R / 64 us / S in S parts; writing and joining them moves 8 S E n k
// bytes, at about 6 bytes a picosecond.  The S that makes the sum of the two
// smallest is the root of their ratio.  Measured, one part against the rule's
// choice and twice it: 20000 rows of one expert, 1024 x 1024, 390 / 60 / 62 us;
// 16384 rows of two, 2048 x 1024, 170 / 79 / 79; 20000 rows of four, 2048 x 256,
// 109 / 43 / 46.  The rows are the capacity's: sums are cut for rows that a larger
// buffer does not hold (1024 live rows, 8 x 1024 x 1024, 12.9 us in a buffer of
// 1920 rows, 32.5 with 64 MB of parts in one of 33664).
int wgrad_splits(int64_t capacity, int n, int k, int num_experts) {
  if (tile_of(capacity, n, k, num_experts) < 256) return 1;
  const int64_t tiles = tiles_of(n, k, num_experts, 256), rows = capacity / num_experts;
  if (tiles * 2 > kFullTiles) return 1;
  const double best =
      sqrt((double)rows / 64.0 * 0.75e6 / ((double)num_experts * (double)n * (double)k));
  const int64_t s = min((int64_t)best, min(kFullTiles / tiles, rows / (4 * kStep)));
  return s > 1 ? (int)s : 1;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_grouped_wgrad_workspace_bytes(int64_t capacity, int n, int k,
                                                    int num_experts) {
  if (check_backward_sizes(capacity, n, k, num_experts, MOE_MIN_ALIGN) != MOE_OK) return 0;
  const int splits = wgrad_splits(capacity, n, k, num_experts);
  return splits > 1 ? (size_t)splits * num_experts * n * k * sizeof(float) : 0;
}

extern "C" moe_status moe_grouped_wgrad_bf16(const void* dy, const void* x, const int32_t* psum,
                                             const int32_t* status, int64_t capacity, int n,
                                             int k, int num_experts, int align, moe_grad_fmt fmt,
                                             int accumulate, void* dw, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  const moe_status c = check_backward_sizes(capacity, n, k, num_experts, align);
  if (c != MOE_OK) return c;
  if (fmt != MOE_GRAD_BF16 && fmt != MOE_GRAD_F32) return MOE_ERR_UNSUPPORTED;
  if (!psum || !status || !dw) return MOE_ERR_NULL;
  if (capacity > 0 && (!dy || !x)) return MOE_ERR_NULL;
  if (((uintptr_t)dy % 16) || ((uintptr_t)x % 16) || ((uintptr_t)dw % 16))
    return MOE_ERR_ALIGNMENT;
  const int splits = wgrad_splits(capacity, n, k, num_experts);
  if (splits > 1) {
    if (!workspace ||
        workspace_bytes < moe_grouped_wgrad_workspace_bytes(capacity, n, k, num_experts))
      return MOE_ERR_WORKSPACE;
    if ((uintptr_t)workspace % 256) return MOE_ERR_ALIGNMENT;
  }
  const int64_t a = capacity * n * 2, b = capacity * k * 2;
  const int64_t out = (int64_t)num_experts * n * k * (fmt == MOE_GRAD_F32 ? 4 : 2);
  const int64_t part = splits > 1 ? (int64_t)splits * num_experts * n * k * 4 : 0;
  if (overlap(dw, out, dy, a) || overlap(dw, out, x, b) || overlap(dw, out, workspace, part) ||
      overlap(workspace, part, dy, a) || overlap(workspace, part, x, b))
    return MOE_ERR_UNSUPPORTED;
  const int tile = tile_of(capacity, n, k, num_experts);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (tile == 64)
    return launch_wgrad_narrow(dy, x, psum, status, capacity, n, k, num_experts, align, fmt,
                               accumulate, dw, st);
  const int64_t items = tiles_of(n, k, num_experts, tile) * splits;
  int64_t grid = device_cus();  // one workgroup per CU, a whole number per XCD
  if (grid > items) grid = items;
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  const bool f32 = fmt == MOE_GRAD_F32;
  auto pick = [&](auto t) {
    constexpr int T = decltype(t)::value;
    return f32 ? (accumulate ? wgrad_kernel<T, true, true, false>
                             : wgrad_kernel<T, true, false, false>)
               : (accumulate ? wgrad_kernel<T, false, true, false>
                             : wgrad_kernel<T, false, false, false>);
  };
  auto kern = splits > 1    ? wgrad_kernel<256, true, false, true>
              : tile == 128 ? pick(std::integral_constant<int, 128>())
                            : pick(std::integral_constant<int, 256>());
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0, st, (const uint8_t*)dy,
                     (const uint8_t*)x, psum, status, capacity, n, k, num_experts, align,
                     splits, splits > 1 ? workspace : dw);
  if (splits > 1) {
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH;
    const int64_t count = (int64_t)num_experts * n * k;
    auto join = f32 ? wgrad_join_kernel<true> : wgrad_join_kernel<false>;
    hipLaunchKernelGGL(join, dim3((unsigned)((count + 8 * kJoinThreads - 1) / (8 * kJoinThreads))),
                       dim3(kJoinThreads), 0, st,
                       (const float*)workspace, splits, count, accumulate, dw);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
