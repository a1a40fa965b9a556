// moe_silu_mul_bf16_backward: gradient of y = silu(g) * u for every live
// expanded row.
//
// With s = 1 / (1 + exp(-g)) and silu(g) = g * s:
//   d silu / d g = s + g * s * (1 - s) = s * (1 + g * (1 - s))
//   d g = dy * u * that,   d u = dy * g * s
// For large negative g, exp(-g) is infinite, s is 0 and both gradients are 0;
// for large positive g, s is 1: no case divides by zero.
//
// HBM-bound: three bf16 values read and two written per element of a row.  A
// power-of-two number of threads shares a row, 8 columns (16 bytes) each per
// pass, so short rows fill a workgroup several at a time.  A row's data is
// loaded before its label is known (the row lies below the total, so the
// loads are in bounds; an alignment pad's values are dropped): one memory
// round trip per row instead of three.  Loads and stores pass the caches by
// (nothing here is read twice): 18432 rows of I = 2048 take 61.8 us, 6.1 TB/s,
// against 67.2 with plain ones; a backward pass around it takes the same time
// with both.
#include "common.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct Grad2 {
  float dg, du;
};
__device__ __forceinline__ Grad2 silu_mul_grad(float g, float u, float dy) {
  const float s = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-g)));
  return {dy * u * (s * (1.0f + g * (1.0f - s))), dy * (g * s)};
}

__global__ __launch_bounds__(kThreads) void silu_backward_kernel(
    const uint16_t* gu, const uint16_t* __restrict__ dy, const int32_t* __restrict__ m_indices,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity,
    int inter, int E, int row_shift, uint16_t* dgu) {
  const int rows_per_block = kThreads >> row_shift, tpr = 1 << row_shift;
  const int tc = threadIdx.x & (tpr - 1), tr = threadIdx.x >> row_shift;
  const int64_t nrows = min((int64_t)status[0], capacity);
  for (int64_t m = (int64_t)blockIdx.x * rows_per_block + tr; m < nrows;
       m += (int64_t)gridDim.x * rows_per_block) {
    const int e = m_indices[m];
    const uint16_t* grow = gu + m * (2 * (int64_t)inter);
    const uint16_t* yrow = dy + m * (int64_t)inter;
    uint16_t* drow = dgu + m * (2 * (int64_t)inter);
    bool live = false, known = false;
    for (int c = tc * 8; c < inter; c += tpr * 8) {
      const u32x4 gv = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(grow + c));
      const u32x4 uv =
          __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(grow + inter + c));
      const u32x4 yv = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(yrow + c));
      if (!known) {
        live = e >= 0 && e < E && m < psum[e];
        known = true;
      }
      if (!live) break;
      u32x4 og, ou;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Grad2 a = silu_mul_grad(__uint_as_float(gv[i] << 16), __uint_as_float(uv[i] << 16),
                                      __uint_as_float(yv[i] << 16));
        const Grad2 b = silu_mul_grad(__uint_as_float(gv[i] & 0xffff0000u),
                                      __uint_as_float(uv[i] & 0xffff0000u),
                                      __uint_as_float(yv[i] & 0xffff0000u));
        og[i] = (uint32_t)f32_to_bf16_rne(a.dg) | ((uint32_t)f32_to_bf16_rne(b.dg) << 16);
        ou[i] = (uint32_t)f32_to_bf16_rne(a.du) | ((uint32_t)f32_to_bf16_rne(b.du) << 16);
      }
      __builtin_nontemporal_store(og, reinterpret_cast<u32x4*>(drow + c));
      __builtin_nontemporal_store(ou, reinterpret_cast<u32x4*>(drow + inter + c));
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_silu_mul_bf16_backward(const void* gate_up, const void* dy,
                                                 const int32_t* m_indices, const int32_t* psum,
                                                 const int32_t* status, int64_t capacity,
                                                 int inter, int num_experts, int align,
                                                 void* d_gate_up, void* stream) {
  if (capacity < 0 || capacity > (1LL << 30) || inter <= 0 || inter % 8 != 0 ||
      num_experts < 1 || num_experts > MOE_MAX_EXPERTS)
    return MOE_ERR_SHAPE;
  if (align < MOE_MIN_ALIGN || align > MOE_MAX_ALIGN || (align & (align - 1)))
    return MOE_ERR_UNSUPPORTED;
  if (capacity % align != 0) return MOE_ERR_SHAPE;
  if (!m_indices || !psum || !status) return MOE_ERR_NULL;
  if (capacity > 0 && (!gate_up || !dy || !d_gate_up)) return MOE_ERR_NULL;
  if (((uintptr_t)gate_up % 16) || ((uintptr_t)dy % 16) || ((uintptr_t)d_gate_up % 16))
    return MOE_ERR_ALIGNMENT;
  if (capacity == 0) return MOE_OK;
  const int64_t row = capacity * (int64_t)inter * 2;
  if ((d_gate_up != gate_up && overlap(d_gate_up, 2 * row, gate_up, 2 * row)) ||
      overlap(d_gate_up, 2 * row, dy, row))
    return MOE_ERR_UNSUPPORTED;
  int row_shift = 0;  // threads per row: a power of two that covers the row, at most all
  while ((8 << row_shift) < inter && (1 << row_shift) < kThreads) ++row_shift;
  const int64_t rows_per_block = kThreads >> row_shift;
  const int64_t blocks = (capacity + rows_per_block - 1) / rows_per_block;
  const int64_t grid = blocks < 16384 ? blocks : 16384;  // grid-stride over the rest
  hipLaunchKernelGGL(silu_backward_kernel, dim3((unsigned)grid), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), (const uint16_t*)gate_up,
                     (const uint16_t*)dy, m_indices, psum, status, capacity, inter, num_experts,
                     row_shift, (uint16_t*)d_gate_up);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
