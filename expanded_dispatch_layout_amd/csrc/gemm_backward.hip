// Gradients of the grouped bf16 GEMM out[m, :] = a[m, :] . w[e]^T over the
// expanded rows:
//   moe_grouped_dgrad_bf16   dx[m, t]    = sum_j dy[m, j] w[e, j, t]
//   moe_grouped_wgrad_bf16   dw[e, j, t] = sum_m dy[m, j] x[m, t], m over e's
//                                          live rows
//
// 64 x 64 tiles through LDS, four waves of one 16-row band each,
// v_mfma_f32_16x16x32_bf16.  An operand whose reduction axis is not the
// contiguous one is transposed on its way into LDS.
#include "gemm_backward.hpp"

namespace moe {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int T = 64;         // tile edge, and the reduction step
constexpr int LD = T + 8;     // LDS row pitch (16-byte aligned rows)

// acc[j] += A-tile (16 rows from row0) x B-tile^T, both [64][T] in LDS with
// the reduction axis contiguous.
__device__ __forceinline__ void tile_mma(const uint16_t (*A)[LD], const uint16_t (*B)[LD],
                                         int row0, int lane, v4f (&acc)[4]) {
  const int f = lane & 15, g = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bf16x8 a = *reinterpret_cast<const bf16x8*>(&A[row0 + f][h * 32 + g * 8]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 b = *reinterpret_cast<const bf16x8*>(&B[j * 16 + f][h * 32 + g * 8]);
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc[j], 0, 0, 0);
    }
  }
}

// 64 rows x 64 columns of a row-major matrix, rows from src (pitch ld); rows
// >= nr and columns >= nc read as 0.
template <bool kTranspose>
__device__ __forceinline__ void load_tile(const uint16_t* src, int64_t ld, int nr, int nc,
                                          uint16_t (*dst)[LD]) {
  for (int c = threadIdx.x; c < T * T / 8; c += kThreads) {
    const int r = c / (T / 8), q = (c % (T / 8)) * 8;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (r < nr && q < nc) v = *reinterpret_cast<const u32x4*>(src + r * ld + q);
    if constexpr (kTranspose) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dst[q + 2 * i][r] = (uint16_t)(v[i] & 0xffffu);
        dst[q + 2 * i + 1][r] = (uint16_t)(v[i] >> 16);
      }
    } else {
      *reinterpret_cast<u32x4*>(&dst[r][q]) = v;
    }
  }
}

// Live rows [st, en) of expert e.
__device__ __forceinline__ void expert_rows(const int32_t* psum, int64_t nrows, int align, int e,
                                            int64_t& st, int64_t& en) {
  st = e ? max(0, align_up_i(psum[e - 1], align)) : 0;
  en = min((int64_t)psum[e], nrows);
}

__global__ __launch_bounds__(kThreads) void dgrad_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ w,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, uint16_t* __restrict__ dx) {
  __shared__ __attribute__((aligned(16))) uint16_t A[T][LD], B[T][LD];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int64_t nrows = min((int64_t)status[0], capacity);
  // Row tile blockIdx.x of the experts' blocks, counted expert by expert.
  int64_t left = blockIdx.x, st = 0, en = 0;
  int e = 0;
  for (; e < E; ++e) {
    expert_rows(psum, nrows, align, e, st, en);
    const int64_t tiles = en > st ? (en - st + T - 1) / T : 0;
    if (left < tiles) break;
    left -= tiles;
  }
  if (e == E) return;
  const int64_t m0 = st + left * T;
  const int live = (int)min((int64_t)T, en - m0);
  const int t0 = blockIdx.y * T;
  v4f acc[4] = {};
  for (int j0 = 0; j0 < n; j0 += T) {
    load_tile<false>(dy + m0 * n + j0, n, live, T, A);
    load_tile<true>(w + ((int64_t)e * n + j0) * k + t0, k, T, T, B);
    __syncthreads();
    tile_mma(A, B, wid * 16, lane, acc);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = wid * 16 + (lane >> 4) * 4 + q;
      if (r < live) dx[(m0 + r) * k + t0 + j * 16 + (lane & 15)] = f32_to_bf16_rne(acc[j][q]);
    }
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
  const dim3 grid((unsigned)((capacity + T - 1) / T + num_experts), (unsigned)(k / T));
  hipLaunchKernelGGL(dgrad_kernel, grid, dim3(kThreads), 0, reinterpret_cast<hipStream_t>(stream),
                     (const uint16_t*)dy, (const uint16_t*)w, psum, status, capacity, n, k,
                     num_experts, align, (uint16_t*)dx);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
