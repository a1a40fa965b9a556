// What the grouped products' gradients share.
#pragma once

#include "lds_dma.hpp"

namespace moe {

constexpr int kMaxBlocks64 = 511;  // n / 64 and k / 64, as the forward GEMM's k

inline moe_status check_backward_sizes(int64_t capacity, int n, int k, int num_experts,
                                       int align) {
  if (capacity < 0 || capacity > (1LL << 30) || n <= 0 || k <= 0 || n % 128 || k % 64 ||
      num_experts < 1 || num_experts > MOE_MAX_EXPERTS)
    return MOE_ERR_SHAPE;
  if (align < MOE_MIN_ALIGN || align > MOE_MAX_ALIGN || (align & (align - 1)))
    return MOE_ERR_UNSUPPORTED;
  if (capacity % align != 0) return MOE_ERR_SHAPE;
  if (n / 64 > kMaxBlocks64 || k / 64 > kMaxBlocks64) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

typedef float v4f __attribute__((ext_vector_type(4)));

// This workgroup's item of the round that starts at item `base` (nitems: none).
// Neighbouring items go to the workgroups of one XCD, whose L2 they share, and
// every XCD gets as many: the grid is a bound, and rounds that are not full
// would otherwise leave whole XCDs idle (64 rows per expert, 8 x 2048 x 1024:
// 22.4 -> 13.0 us; 1024 rows per expert, in a round and a fifth: 56 -> 51).
__device__ __forceinline__ uint32_t round_item(uint32_t base, uint32_t nitems) {
  const uint32_t left = nitems > base ? nitems - base : 0;
  const uint32_t per = (min(left, gridDim.x) + kXcds - 1) / kXcds;
  const uint32_t slot = blockIdx.x / kXcds;
  return slot < per ? min(base + blockIdx.x % kXcds * per + slot, nitems) : nitems;
}

__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]),
               pk_bf16(v[6], v[7])};
}

// 8 consecutive gradients to dw (fp32 or bf16), added to what is there.
template <bool kF32>
__device__ __forceinline__ void store_grad8(void* dw, int64_t at, const float (&v)[8],
                                            int accumulate) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[i];
  if constexpr (kF32) {
    v4f* o = reinterpret_cast<v4f*>((float*)dw + at);
    v4f lo = {r[0], r[1], r[2], r[3]}, hi = {r[4], r[5], r[6], r[7]};
    if (accumulate) {
      lo += o[0];
      hi += o[1];
    }
    o[0] = lo;
    o[1] = hi;
  } else {
    u32x4* o = reinterpret_cast<u32x4*>((uint16_t*)dw + at);
    if (accumulate) {
      const u32x4 q = *o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[2 * i] += __uint_as_float(q[i] << 16);
        r[2 * i + 1] += __uint_as_float(q[i] & 0xffff0000u);
      }
    }
    *o = pack8(r);
  }
}

// Launches of grad_narrow.hip.
constexpr int kNarrowTile = 64;
moe_status launch_dgrad_narrow(const void* dy, const void* w, const int32_t* psum,
                               const int32_t* status, int64_t capacity, int n, int k,
                               int num_experts, int align, void* dx, hipStream_t s);
moe_status launch_wgrad_narrow(const void* dy, const void* x, const int32_t* psum,
                               const int32_t* status, int64_t capacity, int n, int k,
                               int num_experts, int align, moe_grad_fmt fmt, int accumulate,
                               void* dw, hipStream_t s);

}  // namespace moe
