// moe_gather_backward: gradient of the combine out[r] = f * sum_k c[r,k] *
// D[dst(r,k)].
//
//   d D[dst(r,k)] = (f * c[r,k]) * dout[r]
//   d c[r,k]      = f * <dout[r], D[dst(r,k)]>
//
// HBM-bound: each expert row is read and written once.  One wave per slot
// (r, k): it reads dout[r] and its expert row 16 bytes per lane at a time and
// writes its gradient row, and the 64 lanes' partial products are summed in a
// fixed order.  The slots of a token are neighbouring waves, so dout[r] comes
// from HBM once and from the caches for its other slots; there is nothing to
// join between waves, and a token's slots run side by side however few tokens
// there are.  4096 tokens of H = 7168 with 8 slots each: 205 us, 4.9 TB/s, the
// rate of a plain copy.  (Loads and stores that pass the caches by take 191,
// but then the products that read the gradient rows next take 10 us longer in
// all.)
#include "common.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

template <bool kDots>
__global__ __launch_bounds__(kThreads) void gather_backward_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ eo,
    const int32_t* __restrict__ src2dst, const float* __restrict__ topk_w, float factor,
    const int32_t* __restrict__ psum_rank, int nsrc, int64_t rows, int hidden, int topk,
    int64_t capacity, uint16_t* __restrict__ deo, float* __restrict__ dw) {
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nslots = valid_rows(psum_rank, nsrc, rows) * topk;
  for (int64_t s = (int64_t)blockIdx.x * kWaves + wid; s < nslots;
       s += (int64_t)gridDim.x * kWaves) {
    const int d = src2dst[s];
    const float wk = topk_w ? topk_w[s] : 1.f;
    if (d < 0 || d >= capacity) {
      if (kDots && lane == 0) dw[s] = 0.f;
      continue;
    }
    const float c = __fmul_rn(factor, wk);
    const uint16_t* orow = dout + (s / topk) * hidden;
    const uint16_t* erow = eo + (int64_t)d * hidden;
    uint16_t* drow = deo + (int64_t)d * hidden;
    float dot = 0.f;
    for (int h = lane * 8; h < hidden; h += kWave * 8) {
      const u32x4 ov = *reinterpret_cast<const u32x4*>(orow + h);
      u32x4 ev;
      if constexpr (kDots) ev = *reinterpret_cast<const u32x4*>(erow + h);
      u32x4 g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(ov[i] << 16);
        const float hi = __uint_as_float(ov[i] & 0xffff0000u);
        if constexpr (kDots) {
          dot += lo * __uint_as_float(ev[i] << 16);
          dot += hi * __uint_as_float(ev[i] & 0xffff0000u);
        }
        g[i] = (uint32_t)f32_to_bf16_rne(__fmul_rn(c, lo)) |
               ((uint32_t)f32_to_bf16_rne(__fmul_rn(c, hi)) << 16);
      }
      *reinterpret_cast<u32x4*>(drow + h) = g;
    }
    if constexpr (kDots) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
      if (lane == 0) dw[s] = __fmul_rn(factor, dot);
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_gather_backward(const void* dout, const void* expert_out,
                                          const int32_t* src2dst, const float* topk_weights,
                                          float routed_scaling_factor,
                                          const int32_t* psum_recv_per_rank, int num_src_ranks,
                                          int64_t rows, int hidden, int topk, int64_t capacity,
                                          void* d_expert_out, float* d_topk_weights,
                                          void* stream) {
  if (rows < 0 || hidden <= 0 || hidden % kGroup != 0 || topk < 1 || topk > MOE_MAX_TOPK ||
      capacity < 0 || rows > (1LL << 30))
    return MOE_ERR_SHAPE;
  if (num_src_ranks < 0 || (psum_recv_per_rank && num_src_ranks == 0)) return MOE_ERR_SHAPE;
  if (rows > 0 && (!src2dst || !dout)) return MOE_ERR_NULL;
  if (!(routed_scaling_factor == routed_scaling_factor) ||
      __builtin_isinf(routed_scaling_factor))
    return MOE_ERR_UNSUPPORTED;  // a NaN or infinite factor
  if (capacity > 0 && (!d_expert_out || (d_topk_weights && !expert_out))) return MOE_ERR_NULL;
  if (((uintptr_t)dout % 16) || ((uintptr_t)expert_out % 16) || ((uintptr_t)d_expert_out % 16) ||
      ((uintptr_t)d_topk_weights % 4))
    return MOE_ERR_ALIGNMENT;
  if (hidden > 8192) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const int64_t out = capacity * hidden * 2, weights = rows * topk * 4;
  if (overlap(d_expert_out, out, dout, rows * hidden * 2) ||
      overlap(d_expert_out, out, d_topk_weights ? expert_out : nullptr, out) ||
      overlap(d_expert_out, out, src2dst, weights) ||
      overlap(d_expert_out, out, topk_weights, weights) ||
      overlap(d_topk_weights, weights, dout, rows * hidden * 2) ||
      overlap(d_topk_weights, weights, expert_out, out) ||
      overlap(d_topk_weights, weights, d_expert_out, out) ||
      overlap(d_topk_weights, weights, src2dst, weights) ||
      overlap(d_topk_weights, weights, topk_weights, weights))
    return MOE_ERR_UNSUPPORTED;
  const int64_t blocks = (rows * topk + kWaves - 1) / kWaves;
  const int64_t grid = blocks < 65536 ? blocks : 65536;  // grid-stride over the rest
  auto kern = d_topk_weights ? gather_backward_kernel<true> : gather_backward_kernel<false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), (const uint16_t*)dout,
                     (const uint16_t*)expert_out, src2dst, topk_weights, routed_scaling_factor,
                     psum_recv_per_rank, num_src_ranks, rows, hidden, topk, capacity,
                     (uint16_t*)d_expert_out, d_topk_weights);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
