// moe_grouped_wgrad_bf16: weight gradient of the grouped bf16 GEMM,
//   dw[e, j, t] = sum over the live rows m of expert e of dy[m, j] * x[m, t].
#include "gemm_backward.hpp"
#include "lds_dma.hpp"

namespace moe {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int TN = 256, TK = 256;            // output tile: dy columns x x columns
constexpr int kStep = 32;                    // rows per stage
constexpr int kRowBytes = 512;               // 256 bf16
constexpr int kOpBytes = kStep * kRowBytes;  // 16 KB: one operand of a stage
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kStages = 5;
constexpr int kRing = kStages * kStageBytes;   // 128 KB
constexpr int kLds = kRing; // 160 KB
constexpr int kLoads = 4;                      // DMA instructions per wave and stage
constexpr int FI = 8, FJ = 4;                  // 16-wide tiles per wave: 128 x columns, 64 dy ones

constexpr int64_t kMinTiles = 256;
constexpr int64_t kMaxSplitTiles = 512;

struct Tile {
  int e, j0, t0;
  int64_t st;  // first row
  int live;    // rows
};

// Items of one expert: panels of 8 tiles along t, j-major inside a panel, so
// that the 32 neighbouring items of an XCD's CUs are a 4 x 8 block and share
// their operands in its L2.
__device__ __forceinline__ Tile decode(int64_t item, int NJ, int NT, const int32_t* psum,
                                       int64_t nrows, int align) {
  Tile t;
  const int per = NJ * NT;
  t.e = (int)(item / per);
  const int local = (int)(item % per);
  const int panel = local / (8 * NJ);
  const int rem = local - panel * 8 * NJ;
  const int w = min(8, NT - panel * 8);
  t.j0 = rem / w * TN;
  t.t0 = (panel * 8 + rem % w) * TK;
  t.st = t.e ? max(0, align_up_i(psum[t.e - 1], align)) : 0;
  const int64_t en = min((int64_t)psum[t.e], nrows);
  t.live = en > t.st ? (int)(en - t.st) : 0;
  return t;
}

// Stages of a tile: computed in pairs, so an odd count gets one of zeros.
__device__ __forceinline__ int stages_of(int live) {
  return 2 * ((live + 2 * kStep - 1) / (2 * kStep));
}

template <bool kF32>
__global__ __launch_bounds__(kThreads, 1) void wgrad_kernel(
    const uint8_t* __restrict__ dy, const uint8_t* __restrict__ x,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, int accumulate, void* __restrict__ dw) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];  // addresses are XORed
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = lds_addr(lds);
  const int64_t nrows = min((int64_t)status[0], capacity);
  const int NJ = (n + TN - 1) / TN, NT = (k + TK - 1) / TK;
  const int64_t nitems = (int64_t)E * NJ * NT;
  const int per_xcd = gridDim.x / kXcds;
  const int64_t first = (int64_t)(blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;

  // Fragment addresses within a stage: tile i of a wave is its 32-byte piece
  // i ^ key of a row, so one lane base serves all of them through an XOR.
  const int wj = wid >> 1, wt = wid & 1;
  uint32_t fx, fy;  // x, dy
  {
    const uint32_t base = lds0 + tr_lane_offset(lane);
    fx = base + kOpBytes + wt * 256;
    fy = (base + (wj >> 1) * 256) ^ (uint32_t)((wj & 1) * FJ * 32);
  }

  // DMA side: the next stage to load.
  int64_t d_item = first;
  int d_left = 0;    // rows left of its tile (<= 0: a stage of zeros)
  int d_stages = 0;  // stages left of its tile
  const uint8_t *d_dy = nullptr, *d_x = nullptr;
  uint32_t d_offa[2], d_offb[2];  // x, dy: offsets of this lane's chunks
  uint32_t d_slot = 0;            // LDS offset of the next slot
  auto d_open = [&]() __attribute__((always_inline)) {  // next tile that has rows
    while (d_item < nitems) {
      const Tile t = decode(d_item, NJ, NT, psum, nrows, align);
      if (t.live > 0) {
        d_left = t.live;
        d_stages = stages_of(t.live);
        d_dy = dy + (t.st * n + t.j0) * 2;
        d_x = x + (t.st * k + t.t0) * 2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = (wid * 2 + j) * 2 + (lane >> 5);
          const int col = ((lane & 31) ^ (tr_key(row) << 1)) * 8;
          d_offb[j] = (uint32_t)(row * n + min(col, n - 8 - t.j0)) * 2u;
          d_offa[j] = (uint32_t)(row * k + min(col, k - 8 - t.t0)) * 2u;
        }
        return;
      }
      d_item += gridDim.x;
    }
  };
  // Load q (0..3) of the next stage: dy rows first, then x.  Rows past the
  // tile's last live one, and every row once there is no tile left, read
  // zeros, so that each step issues the same loads without a branch.
  const int d_row = wid * 4 + (lane >> 5);  // this lane's row in load 0; 2 more per load
  auto d_load = [&](int q) __attribute__((always_inline)) {
    const int j = q & 1;
    const uint8_t* p = q < 2 ? d_dy + d_offb[j] : d_x + d_offa[j];
    p = d_row + 2 * j < d_left ? p : zero_chunk();
    dma16_ptr(p, lds0 + d_slot + wid * 2048 + (q < 2 ? 0 : kOpBytes) + j * 1024);
  };
  auto d_advance = [&]() __attribute__((always_inline)) {
    d_slot = d_slot + kStageBytes == kRing ? 0 : d_slot + kStageBytes;
    d_left -= kStep;
    d_dy += (int64_t)kStep * n * 2;
    d_x += (int64_t)kStep * k * 2;
    if (--d_stages <= 0 && d_item < nitems) {
      d_item += gridDim.x;
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

  for (int64_t item = first; item < nitems; item += gridDim.x) {
    const Tile t = decode(item, NJ, NT, psum, nrows, align);
    const int steps = stages_of(t.live);
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
            if (u % 2 == 0 && u / 2 < FJ) b[h ^ 1][u / 2] = frag_tr<kRowBytes>(ny ^ ((u / 2) << 5));
            else if (u % 2 == 0 && u / 2 < FJ + FI)
              a[h ^ 1][u / 2 - FJ] = frag_tr<kRowBytes>(nx ^ ((u / 2 - FJ) << 5));
            else if (u % 4 == 1 && u / 4 < kLoads) d_load(u / 4);
            sched_fence();
          }
          c_slot = nslot;
          d_advance();
        }
      }
    } else if (accumulate) {
      continue;
    }
    // Epilogue: lane holds t = 4 (lane / 16) + 0..3 of tile i, j = lane % 16 of
    // tile j.
    const int jc = t.j0 + wj * 64, tc = t.t0 + wt * 128 + (lane >> 4) * 4;
    if (jc < n) {
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int64_t row = ((int64_t)t.e * n + jc + j * 16 + (lane & 15)) * k + tc;
#pragma unroll
        for (int i = 0; i < FI; ++i) {
          if (t.t0 + wt * 128 + i * 16 < k) {
            v4f v = acc[i][j];
            if constexpr (kF32) {
              v4f* o = reinterpret_cast<v4f*>((float*)dw + row + i * 16);
              if (accumulate) v += *o;
              *o = v;
            } else {
              uint2* o = reinterpret_cast<uint2*>((uint16_t*)dw + row + i * 16);
              if (accumulate) {
                const uint2 q = *o;
                v += v4f{__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u),
                         __uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u)};
              }
              *o = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
            }
          }
        }
      }
    }
  }
  wait_vmcnt<0>();  // no load may land after the workgroup's LDS has been given away
}

}  // namespace
}  // namespace moe

using namespace moe;

namespace moe {
namespace {

int64_t wide_tiles(int n, int k, int num_experts) {
  return (int64_t)num_experts * ((n + TN - 1) / TN) * ((k + TK - 1) / TK);
}

// Parts that each expert's sum is cut into.  Only the narrow tiles are split,
// where they leave workgroups to spare, and at most so that a wave keeps two
// stages of an average expert's rows.
int wgrad_splits(int64_t capacity, int n, int k, int num_experts) {
  if (wide_tiles(n, k, num_experts) >= kMinTiles) return 1;
  const int64_t tiles = (int64_t)num_experts * (n / kNarrowTile) * (k / kNarrowTile);
  const int64_t by_rows = capacity / num_experts / (8 * kStep * 2);
  const int64_t s = min(kMaxSplitTiles / tiles, by_rows);
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
  const int64_t items = wide_tiles(n, k, num_experts);
  if (items < kMinTiles)
    return launch_wgrad_narrow(dy, x, psum, status, capacity, n, k, num_experts, align, fmt,
                               accumulate, splits, dw, workspace,
                               reinterpret_cast<hipStream_t>(stream));
  int64_t grid = device_cus();  // one workgroup per CU, a whole number per XCD
  if (grid > items) grid = items;
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  auto kern = fmt == MOE_GRAD_F32 ? wgrad_kernel<true> : wgrad_kernel<false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), (const uint8_t*)dy, (const uint8_t*)x,
                     psum, status, capacity, n, k, num_experts, align, accumulate, dw);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
