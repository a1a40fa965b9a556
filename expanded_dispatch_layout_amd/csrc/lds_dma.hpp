// Device helpers of the kernels that stream operands HBM -> LDS directly and
// order those loads themselves.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace moe {

constexpr int kXcds = 8;       // MI355X: 8 XCDs, workgroups dispatched round-robin

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

// 16 bytes of zeros, as a source of dma16_ptr.
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};
__device__ __forceinline__ const uint8_t* zero_chunk() { return (const uint8_t*)kZeros; }

// Fragments of an operand that is staged with its reduction axis along the
// rows (a multiple of 256 bytes each).  A fragment
// (16 columns x 32 rows) is read through ds_read_b64_tr_b16, which gives lane
// l of a 16-lane group column l of 4 rows x 16 columns.  Group g = lane / 16
// reads rows 8 g + 0..3 and then 8 g + 4..7, so that each lane holds 8
// consecutive rows of its column, the order in which the MFMA takes them.
// The 32-byte pieces of a row (16 columns each) are XOR-swizzled within 256
// bytes by tr_key(row), which differs over the 8 rows that half a wave reads
// at once: no bank conflicts (counted: none).
__device__ __forceinline__ int tr_key(int row) { return (row & 3) | (((row >> 3) & 1) << 2); }
// This lane's address of piece 0; piece p of the same 256 bytes is at ^ (p << 5).
template <int kRowBytes>
__device__ __forceinline__ uint32_t tr_lane_offset(int lane) {
  const int row = 8 * (lane >> 4) + ((lane & 15) >> 2), q = lane & 3;
  return (uint32_t)(row * kRowBytes + tr_key(row) * 32 + (q >> 1) * 16 + (q & 1) * 8);
}
template <int kRowBytes>
__device__ __forceinline__ auto frag_tr(uint32_t addr) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) s16x4* lds_p;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(size_t)addr);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(size_t)(addr + 4 * kRowBytes));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Two 16x16 MFMA results that are neighbours along their rows: lane l holds
// rows 4 (l / 16) + 0..3 of column l % 16 of each.  With register r of both
// swapped for every r, lane l holds rows 8 ((l / 16) % 2) + 0..3 (in x) and
// + 4..7 (in y) of tile l / 32: 8 consecutive values.
__device__ __forceinline__ void swap_tiles(uint32_t& x, uint32_t& y) {
  // x's upper half against y's lower half, then x's odd 16-lane rows against
  // y's even ones.
  const auto h = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  const auto r = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
  x = r[0];
  y = r[1];
}
// The same as bf16: 16 consecutive bytes per lane.
template <typename V4>
__device__ __forceinline__ u32x4 pack_tiles(const V4& x, const V4& y) {
  uint32_t a[2] = {pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3])};
  uint32_t b[2] = {pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3])};
#pragma unroll
  for (int i = 0; i < 2; ++i) swap_tiles(a[i], b[i]);
  return u32x4{a[0], a[1], b[0], b[1]};
}

}  // namespace moe
