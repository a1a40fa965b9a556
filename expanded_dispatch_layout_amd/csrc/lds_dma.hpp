// Device helpers of the kernels that stream operands HBM -> LDS directly and
// order those loads themselves.
#pragma once

#include "common.hpp"

namespace moe {

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(size_t)(__attribute__((address_space(3))) const void*)p);
}

// LDS reads by 32-bit LDS address (keeps addresses in single registers and
// lets constant parts fold into the instruction's offset field).
template <typename T>
__device__ __forceinline__ T lds_load(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(addr);
}
template <typename T>
__device__ __forceinline__ void lds_store(uint32_t addr, T v) {
  *reinterpret_cast<__attribute__((address_space(3))) T*>(addr) = v;
}

// Direct HBM -> LDS loads.  Issued from inline assembly so the compiler does
// not treat them as LDS writes that every later LDS read must wait for: the
// kernel orders them itself (vmcnt waits + s_barrier).  Address = 64-bit
// scalar base + 32-bit per-lane offset; lane i's data lands at lds + i * size,
// the LDS base taken from M0, which the asm names as an input operand so the
// compiler itself writes it and knows it is in use.
// The compiler's hazard pass does not look inside inline assembly, so the asm
// brings the wait states itself: one between a scalar write of M0 and the
// load, five between a vector instruction that writes a scalar register
// (v_readfirstlane) and a load that takes its address from it.  The bases of
// a stage's dma16 loads are held in scalar registers by settled(), which waits
// once for all of them.
// A wave-uniform pointer, held in scalar registers (the loads' base operand).
__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const uint8_t*)(((uint64_t)hi << 32) | lo);
}

// A base for dma16 (wave-uniform by construction).
__device__ __forceinline__ const uint8_t* settled(const uint8_t* p) {
  p = uniform_ptr(p);
  asm volatile("s_nop 4" : "+s"(p));
  return p;
}

__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);  // M0: wave-uniform by construction
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma4(const uint8_t* base, uint32_t off, uint32_t lds) {
  base = uniform_ptr(base);
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}

// The same from a 64-bit address per lane.
__device__ __forceinline__ void dma16_ptr(const uint8_t* p, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
// Keep the compiler's scheduler from moving instructions across this point
// (bounds how far it hoists the next step's fragment reads, and with them
// the registers they occupy).
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }
// All of this wave's LDS reads have returned.
__device__ __forceinline__ void wait_lgkm0() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Wait until at most a * NL of this wave's vector-memory operations are
// outstanding, a in [0, MAXA] at run time (s_waitcnt takes an immediate: a
// short compare chain picks it).
template <int NL, int MAXA>
__device__ __forceinline__ void wait_ahead(int a) {
  if constexpr (MAXA <= 0) {
    wait_vmcnt<0>();
  } else {
    if (a >= MAXA) wait_vmcnt<MAXA * NL>();
    else wait_ahead<NL, MAXA - 1>(a);
  }
}

// Two floats -> packed bf16 pair (low = x), round to nearest even: one
// v_cvt_pk_bf16_f32 on gfx950.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_bf16(float x, float y) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{x, y}, bf16x2_t));
}

}  // namespace moe
