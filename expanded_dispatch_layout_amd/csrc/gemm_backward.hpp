// What the grouped products' gradients share.
#pragma once

#include "common.hpp"

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

// Launches of grad_narrow.hip.
constexpr int kNarrowTile = 64;
moe_status launch_dgrad_narrow(const void* dy, const void* w, const int32_t* psum,
                               const int32_t* status, int64_t capacity, int n, int k,
                               int num_experts, int align, void* dx, hipStream_t s);
moe_status launch_wgrad_narrow(const void* dy, const void* x, const int32_t* psum,
                               const int32_t* status, int64_t capacity, int n, int k,
                               int num_experts, int align, moe_grad_fmt fmt, int accumulate,
                               int splits, void* dw, void* workspace, hipStream_t s);

}  // namespace moe
