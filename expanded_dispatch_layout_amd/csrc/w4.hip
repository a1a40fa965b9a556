// moe_grouped_gemm_w4: grouped products of bf16 rows with 4-bit expert weights.
//
//   out[m, j] = sum over groups g of s[e, j, g] * sum_{t in g} a[m, t] q[e, j, t]
//
// int4: q in [-8, 7], bf16 scales; MXFP4: q an E2M1 value, s = 2^(byte - 127).
//
// One workgroup of eight waves per CU walks the items of the device's layout:
// "narrow" ones of up to 32 rows of an expert, whose time is the weights' stream, and
// "wide" ones of 128 rows or "tall" ones of 256, which feed the matrix cores through LDS.
//
// Codes to bf16, in registers, by each wave that needs them.  MXFP4:
// v_cvt_scalef32_pk_bf16_fp4 makes two values with their scale, exactly (a normal bf16
// number for bytes 2..252).  int4: the codes enter as 8 + q; the product starts from
// -8 * (the rows' own sum) instead of 0, one MFMA with a constant operand for all the
// columns, and is scaled in fp32 once its group is complete.
//
// One token's eight experts, 4096 x 7168, MXFP4: 31 us, 4.0 TB/s (a plain sum over as
// many bytes takes longer).  8192 rows, 8 x 4096 x 7168: MXFP4 413 to 435 us, 1.11 to 1.17
// PFLOP/s; int4 of 128 797 us (half more MFMAs, 8 beside 16, and a quarter of the tile,
// since the scaled sums need the registers).
#include "gemm_backward.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512, kWaves = 8;
constexpr int BK = 128;                   // a block of the narrow path

// The lane's number, formed here and now: not held, nor what is made of it, for longer.
__device__ __forceinline__ int lane_now() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
  return l;
}

// 4 x 4 words between the wave's 16-lane rows: word i of row r <-> word r of
// row i.
__device__ __forceinline__ void exchange(u32x4& d) {
  uint32_t x[4] = {d[0], d[1], d[2], d[3]};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto h = __builtin_amdgcn_permlane32_swap(x[i], x[i + 2], false, false);
    x[i] = h[0];
    x[i + 2] = h[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto h = __builtin_amdgcn_permlane16_swap(x[i], x[i + 1], false, false);
    x[i] = h[0];
    x[i + 1] = h[1];
  }
  d = u32x4{x[0], x[1], x[2], x[3]};
}

// 8 E2M1 codes times a power of two.
__device__ __forceinline__ bf16x8 fp4_values(uint32_t d, float scale) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3));
  return __builtin_bit_cast(bf16x8, r);
}
// 8 int4 codes q as 8 + q.  An E4M3 byte below 16 is that many times 2^-9
// (subnormal up to 7, and on in the first binade), so a half byte with its sign bit
// turned is 8 + q: two values an instruction, as for MXFP4.
__device__ __forceinline__ bf16x8 int4_values(uint32_t d) {
  const uint32_t even = (d & 0x0f0f0f0fu) ^ 0x08080808u;
  const uint32_t odd = ((d >> 4) & 0x0f0f0f0fu) ^ 0x08080808u;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u);  // codes 0..3
  const uint32_t hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);  // codes 4..7
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true));
  return __builtin_bit_cast(bf16x8, r);
}
constexpr uint32_t kMinus8 = 0xc100c100u;  // two bf16 values of -8

// kGroup 0: MXFP4; otherwise int4 with scales per 32, 64 or 128.
template <int kGroup>
struct Scales {  // of one column's 128-deep block
  static constexpr int kBytes = kGroup ? 2 * BK / kGroup : 4;
  uint32_t w[2];
  __device__ __forceinline__ void load(uint32_t lds) {
    if constexpr (kGroup == 0 || kGroup == 64) {
      w[0] = lds_load<uint32_t>(lds);
    } else if constexpr (kGroup == 128) {
      w[0] = lds_load<uint16_t>(lds);
    } else {
      w[0] = lds_load<uint32_t>(lds);
      w[1] = lds_load<uint32_t>(lds + 4);
    }
  }
  __device__ __forceinline__ float get(int i) const {  // group i
    if constexpr (kGroup == 0) return __uint_as_float((w[0] >> (8 * i) & 0xffu) << 23);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};

// ------------------------------------------------------------------ items

constexpr int kNarrowRows = 32, kNarrowCols = 64;  // most rows of a narrow item
constexpr int kTileRows = 128, kTallRows = 256;  // of a wide item
constexpr int kDataBytes = 141 * 1024;

// Narrow items: partial sums of 16 rows by 64 or 128 columns for each wave, then
// two items' scales.
constexpr int kMaxTiles = 8, kPartBytes = kWaves * 16 * (16 * kMaxTiles + 4) * 4;

// The three kinds of items: of 128 rows, of up to 32, of up to 16.
constexpr int kWide = 0, kTwo = 1, kOne = 2;

struct __attribute__((aligned(16))) Item {
  int e, col, live, m0;
};
constexpr int kListed = 64;               // narrow items that a workgroup looks up at once

struct Shared {
  __attribute__((aligned(1024))) uint8_t data[kDataBytes];
  int pe[MOE_MAX_EXPERTS];                // psum
  Item list[kListed];
  int gp[3][MOE_MAX_EXPERTS + 1];         // prefix of each kind's row groups per expert
  int tile;                               // rows of a wide item
};

struct Args {
  const uint8_t *a, *w, *sc;
  int64_t nrows;
  int n, k, E, align;
  uint16_t* out;
  bool fits;                              // a narrow item's scales have room in LDS
};

// First row of expert e, and its live rows.
__device__ __forceinline__ int rows_of(const Shared& sh, const Args& p, int e, int& st) {
  if (e >= p.E) return 0;
  st = e ? max(0, align_up_i(sh.pe[e - 1], p.align)) : 0;
  const int64_t en = min((int64_t)sh.pe[e], p.nrows);
  return en > st ? (int)(en - st) : 0;
}

// The row groups of every kind.  Experts of up to 32 rows are narrow, if the scales of
// their items fit (p.fits: K up to 4736 for int4 of 32, 9472 for MXFP4 and int4 of 64,
// 18944 for int4 of 128; one token's 8 products of 4096 x 9472 and x 9600 in MXFP4: 38 and
// 98 us).  The others
// are all narrow or all wide, by the rounds that the workgroups make of their
// 128-column tiles of 32 or 128 rows, which take about 0.55 and 1.3 us for 128 of the
// reduction (weights of 8 x 4096 x 7168 in MXFP4, narrow / wide: 40 rows each 68 / 82 us,
// 56 rows 93 / 75, 75 rows 93 / 77; 8 x 7168 x 2048 in int4: 40 rows 41 / 63, 56 rows
// 42 / 57, 87 rows 60 / 57; 64 x 1024 x 1024 in MXFP4: 40 rows 27 / 26, 56 rows 37 /
// 25).  A bound on rows alone leaves some experts on either side, and the two halves
// then run one after the other (56 rows and a bound of 64: 98, 47 and 44).
template <int kGroup>
__device__ __forceinline__ void list_items(Shared& sh, const Args& p, int lane) {
  int n32 = 0, n128 = 0, n256 = 0;  // row groups of those (of up to 2^25 rows: enough to tell)
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    int st;
    const int rows = min(rows_of(sh, p, e0 + lane, st), 1 << 25);
    const bool more = rows > kNarrowRows;
    n32 += __builtin_amdgcn_readlane(
        wave_incl_scan_i(more ? (rows + kNarrowRows - 1) / kNarrowRows : 0), 63);
    n128 += __builtin_amdgcn_readlane(
        wave_incl_scan_i(more ? (rows + kTileRows - 1) / kTileRows : 0), 63);
    n256 += __builtin_amdgcn_readlane(
        wave_incl_scan_i(more ? (rows + kTallRows - 1) / kTallRows : 0), 63);
  }
  const int64_t tiles = p.n / 128, grid = gridDim.x;
  const bool narrow =
      p.fits && 5 * ((n32 * tiles + grid - 1) / grid) < 12 * ((n128 * tiles + grid - 1) / grid);
  const int64_t tiles256 = (p.n + 255) / 256;
  // 256 rows by the rounds, too: 9, 16 and 29 are what tiles of 128 x 128, 128 x 256 and
  // 256 x 256 last, also as the parts of a last round (w4_kernel).
  auto rounds = [&](int64_t items, int each, int parts) __attribute__((always_inline)) {
    const int64_t rest = items % grid;
    const int last = rest == 0                             ? 0
                     : parts == 4 && rest * 4 <= grid ? 9
                     : rest * 2 <= grid               ? (parts == 4 ? 16 : 9)
                                                      : each;
    return items / grid * each + last;
  };
  const bool tall = kGroup == 0 && !narrow && n256 * tiles256 >= grid &&
                    rounds(n256 * tiles256, 29, 4) < rounds(n128 * tiles256, 16, 2);
  const int tile = tall ? kTallRows : kTileRows;
  int wide = 0, both = 0;  // both: of 32 rows, and of 16 (<< 16; at most one an expert)
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    int st;
    const int e = e0 + lane, rows = rows_of(sh, p, e, st);
    const bool is_wide = (rows > kNarrowRows || !p.fits) && !narrow;
    const int nw = is_wide ? (rows + tile - 1) / tile : 0;
    const int nb = is_wide   ? 0
                   : rows > 16 ? (rows + kNarrowRows - 1) / kNarrowRows
                               : (rows > 0) << 16;
    const int iw = wave_incl_scan_i(nw), ib = wave_incl_scan_i(nb);
    if (e < p.E) {
      sh.gp[kWide][e] = wide + iw - nw;
      sh.gp[kTwo][e] = (both + ib - nb) & 0xffff;
      sh.gp[kOne][e] = (both + ib - nb) >> 16;
    }
    wide += __builtin_amdgcn_readlane(iw, 63);
    both += __builtin_amdgcn_readlane(ib, 63);
  }
  if (lane == 0) {
    sh.tile = tile;
    sh.gp[kWide][p.E] = wide;
    sh.gp[kTwo][p.E] = both & 0xffff;
    sh.gp[kOne][p.E] = both >> 16;
  }
}

// Item i of a kind: expert by expert, column tile by column tile, the row groups
// innermost: they read the same weights side by side on one XCD.  (i may differ
// between lanes.)
__device__ __forceinline__ Item decode(const Shared& sh, const Args& p, int kind, uint32_t i,
                                       int NT, int cols, int rows) {
  const int q = (int)(i / (uint32_t)NT);
  const int* gp = sh.gp[kind];
  int lo = 0, hi = p.E - 1;  // last e with gp[e] <= q
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gp[mid] <= q) lo = mid;
    else hi = mid - 1;
  }
  const int g0 = gp[lo], ge = gp[lo + 1] - g0;
  const int local = (int)(i - (uint32_t)NT * (uint32_t)g0);
  int st = 0;
  const int all = rows_of(sh, p, lo, st);
  const int at = local % ge * rows;
  return Item{lo, local / ge * cols, min(rows, all - at), st + at};
}
__device__ __forceinline__ Item uniform(const Item& t) {
  return Item{__builtin_amdgcn_readfirstlane(t.e), __builtin_amdgcn_readfirstlane(t.col),
              __builtin_amdgcn_readfirstlane(t.live), __builtin_amdgcn_readfirstlane(t.m0)};
}

// ----------------------------------------------------------------- narrow

// The weights' stream decides.  An item is 16 kMt rows and 16 kTiles cs columns: the
// waves are cs groups of 16 kTiles columns by 8 / cs parts of the reduction, which take
// its 128-deep blocks in turn, straight from memory into registers; the next block is
// asked for, also of the next item, once the present one is used, and the two waves of
// a SIMD take turns (two blocks in flight are no faster, 31.3 us against 31.2 for one
// token's eight products of 4096 x 7168, and four cost 1 us: their code is longer than
// the few steps a wave makes).  The parts' sums meet in LDS, in the parts' order.
// 17 to 32 rows take 128 columns to a wave, so that the rows are read half as often
// (200 rows, 8 x 7168 x 2048, int4: 34 us with 64 columns, 30 so).
// The item's scales are one contiguous piece of memory, copied to LDS during the item
// before it: read where they are needed, 4 bytes of a line at a time, they cost more
// requests than the codes (51 us against 36, at that time).
template <int kGroup, int kMt, int kTiles>
__device__ __forceinline__ void narrow(Shared& sh, const Args& p, uint32_t first_item,
                                       uint32_t last_item, uint32_t nitems, int cs,
                                       uint32_t& base, int lane, int wid) {
  constexpr bool kFp4 = kGroup == 0;
  constexpr int kKind = kMt == 2 ? kTwo : kOne, kCols = 16 * kTiles;  // a wave's columns
  constexpr int kPitch = kCols + 4;                              // of its partial sums
  constexpr int kG = kFp4 ? 1 : 128 / kGroup, kSteps = 4 / kG;   // groups of a block, MFMAs each
  constexpr int kStepLoads = kTiles + 4 * kMt;
  u32x4 wv[kTiles], xv[kMt][4];  // the block loaded
  const int c = lane & 15, qd = lane >> 4;
  const int k = p.k, KB = k / BK, cols = kCols * cs, NT = p.n / cols;
  const int ks = kWaves / cs, cg = wid % cs, kp = wid / cs;
  const int nk = KB > kp ? (KB - kp + ks - 1) / ks : 0;  // blocks of this wave per item
  // Steps of every wave per item: one past its blocks loads one address and adds
  // nothing.
  const int steps = (KB + ks - 1) / ks;
  const int sc_row = KB * Scales<kGroup>::kBytes, sc_bytes = cols * sc_row;
  const uint32_t sc0 = lds_addr(sh.data) + kWaves * 16 * kPitch * 4;
  const uint32_t sc_slot = (uint32_t)(sc_bytes + 1023) & ~1023u;
  const uint32_t sc_lane = sc0 + (uint32_t)((cg * kCols + c) * sc_row);

  int count = 0;  // items in the list
  auto item_of = [&](int i) __attribute__((always_inline)) { return uniform(sh.list[i]); };
  auto copy_scales = [&](int i) __attribute__((always_inline)) {
    if (i >= count) return;
    const Item t = item_of(i);
    const uint8_t* from = p.sc + ((int64_t)t.e * p.n + t.col) * sc_row;
    for (int at = wid * 1024; at < sc_bytes; at += kWaves * 1024)
      dma16_ptr(from + min(at + lane * 16, sc_bytes - 16), sc0 + (i & 1) * sc_slot + at);
  };

  int li = 0, lk = 0;  // loading side: item and step
  const uint8_t *wp, *ap[kMt];
  int64_t w_step, x_step, w_tile;
  auto nothing = [&]() __attribute__((always_inline)) {
    wp = p.w;
#pragma unroll
    for (int m = 0; m < kMt; ++m) ap[m] = p.a;
    w_step = x_step = w_tile = 0;
  };
  auto open = [&]() __attribute__((always_inline)) {
    if (li >= count || nk == 0) {
      nothing();
      return;
    }
    const Item t = item_of(li);
    wp = p.w + ((int64_t)t.e * p.n + t.col + cg * kCols + c) * (k / 2) + 16 * qd +
         kp * (BK / 2);
    // Rows past the live ones repeat the last one: a row of the result comes
    // from its own row of a alone, and theirs are not stored.
#pragma unroll
    for (int m = 0; m < kMt; ++m)
      ap[m] = p.a + ((int64_t)(t.m0 + min(16 * m + c, t.live - 1)) * k + 8 * qd + kp * BK) * 2;
    w_step = ks * (BK / 2);
    x_step = ks * BK * 2;
    w_tile = (int64_t)8 * k;
  };
  auto load = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kTiles; ++j) wv[j] = *reinterpret_cast<const u32x4*>(wp + j * w_tile);
#pragma unroll
    for (int m = 0; m < kMt; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[m][i] = *reinterpret_cast<const u32x4*>(ap[m] + 64 * i);
      ap[m] += x_step;
    }
    wp += w_step;
    if (++lk == nk) nothing();
    if (lk == steps) {
      lk = 0;
      ++li;
      open();
    }
  };
  v4f acc[kMt][kTiles];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
      for (int j = 0; j < kTiles; ++j) acc[m][j] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  auto compute = [&](uint32_t scales) __attribute__((always_inline)) {
    Scales<kGroup> sc[kTiles];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) sc[j].load(scales + (uint32_t)(16 * j * sc_row));
#pragma unroll
    for (int j = 0; j < kTiles; ++j) exchange(wv[j]);
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      if constexpr (!kFp4) sched_fence();  // keeps the groups' values apart
      v4f off[kMt];
      if constexpr (!kFp4) {
        const u32x4 m8 = {kMinus8, kMinus8, kMinus8, kMinus8};
#pragma unroll
        for (int m = 0; m < kMt; ++m) {
          off[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
            off[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, xv[m][g * kSteps + i]),
                __builtin_bit_cast(bf16x8, m8), off[m], 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        if constexpr (kGroup == 32) sched_fence();
        bf16x8 v[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          v[i] = kFp4 ? fp4_values(wv[j][i], sc[j].get(i)) : int4_values(wv[j][g * kSteps + i]);
#pragma unroll
        for (int m = 0; m < kMt; ++m) {
          v4f part = kFp4 ? acc[m][j] : off[m];
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, xv[m][g * kSteps + i]), v[i], part, 0, 0, 0);
          if constexpr (kFp4) acc[m][j] = part;
          else acc[m][j] += part * sc[j].get(g);
        }
      }
    }
  };
  // Sums of the parts, 16 rows at a time.  Lane: rows 4 qd + 0..3 of column 16 j + c.
  float* part = reinterpret_cast<float*>(sh.data);
  auto join = [&](int i) __attribute__((always_inline)) {
    const Item t = item_of(i);
    // This wave's copies of the next item's scales, older than an item's loads,
    // have landed.
    wait_vmcnt<kStepLoads>();
#pragma unroll
    for (int m = 0; m < kMt; ++m) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          part[(wid * 16 + 4 * qd + r) * kPitch + 16 * j + c] = acc[m][j][r];
      wait_lgkm0();
      barrier();
      if (m == 0) copy_scales(i + 2);  // in place of this item's
      const int per = cols / 4;        // 4 columns to a thread
      for (int at = 64 * wid + lane; at < per * min(16, t.live - 16 * m); at += kThreads) {
        const int row = at / per, col = at % per;
        const float* from =
            part + (col / (kCols / 4) * 16 + row) * kPitch + col % (kCols / 4) * 4;
        v4f v = {0.f, 0.f, 0.f, 0.f};
        for (int q = 0; q < ks; ++q)
          v += *reinterpret_cast<const v4f*>(from + q * cs * 16 * kPitch);
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        *reinterpret_cast<u32x2*>(p.out + ((int64_t)t.m0 + 16 * m + row) * p.n + t.col +
                                  col * 4) = u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
      }
      wait_lgkm0();
      barrier();  // the partial sums have been read
    }
  };
  for (;; base += count * gridDim.x) {
    // The next items of this workgroup, looked up by a lane each.
    barrier();  // the list and the scales before have been read
    const uint32_t mine = round_item(base + lane * gridDim.x, nitems);
    const bool here = lane < kListed && mine < last_item;
    count = __popcll(__ballot(here));
    if (count == 0) return;
    if (wid == 0 && here)
      sh.list[lane] = decode(sh, p, kKind, mine - first_item, NT, cols, 16 * kMt);
    wait_lgkm0();
    barrier();
    li = lk = 0;
    open();
    copy_scales(0);
    load();
    wait_vmcnt<kStepLoads>();
    barrier();  // the first scales have landed
    copy_scales(1);
    // The loop has one way out: with one after every step, also unrolled, the compiler
    // joins them into one that leads back to the start, and waits there for the
    // youngest load.
    for (int ci = 0; ci < count; ++ci) {
      uint32_t scales = sc_lane + (uint32_t)(kp * Scales<kGroup>::kBytes) + (ci & 1) * sc_slot;
      clear();
      for (int t = 0; t < steps; ++t) {
        if (t < nk) compute(scales);
        load();
        scales += (uint32_t)(ks * Scales<kGroup>::kBytes);
      }
      join(ci);
    }
  }
}

// ------------------------------------------------------------------- wide

// Rows of 128 bytes: chunks of 16 bytes are XOR-swizzled by bits 2, 1 and 3 of the
// row, so that the 16 lanes that a 16-byte LDS read serves at once fall on different
// banks: 16 consecutive rows, or rows 0-3 and 12-15 with 4-11 of the lanes that read
// two chunks further on.
__device__ __forceinline__ int x_key(int row) {
  return (row >> 2 & 1) | (row & 2) | (row >> 1 & 4);
}
__device__ __forceinline__ void dma4_ptr(const uint8_t* p, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}

// 128 rows, 64 kFn columns: eight waves, 2 by 4, of 64 x 16 kFn.  Waves 4-7
// stream the rows, 64 deep along the reduction at a time, waves 0-3 the codes and
// scales, 128 deep: a stage is one request for each row or column, and requests (4
// bytes of scales, 32 of codes) are what bounds shorter ones (8192 rows, 8 x 4096 x
// 7168, MXFP4: 606 us with 64 for all, 515 so).  A wave computes on 64 from registers
// while it reads the next ones' fragments, a read between any two MFMAs (515 -> 490;
// with 8-byte reads of the codes 474).
template <int kGroup, int kFn>
__device__ __forceinline__ void wide(Shared& sh, const Args& p, const Item& t, int lane,
                                     int wid) {
  constexpr bool kFp4 = kGroup == 0;
  constexpr int kFm = 4, kBn = 64 * kFn;
  // Rows are staged 128 deep, too, where the tile leaves room for it: one barrier for
  // twice the products (800 rows, 8 x 4096 x 7168: 91 -> 80 us).
  constexpr bool kPair = kFn == 2;
  constexpr int kScWords = kGroup == 32 ? 2 : 1;                   // per column and stage
  constexpr int kA = kPair ? 3 : 4, kW = kPair && kScWords == 1 ? 5 : 4;  // stages in LDS
  constexpr int kHalf = kTileRows * 128;                           // rows, 64 deep
  constexpr int kABytes = kPair ? 2 * kHalf : kHalf, kCodeBytes = kBn * 64;  // of a stage
  constexpr int kWBytes = kCodeBytes + kScWords * 1024;
  constexpr int kALoads = kPair ? 8 : 4, kWLoads = kFn + kScWords;  // per wave and stage
  static_assert(kA * kABytes + kW * kWBytes <= kDataBytes);
  const int n = p.n, k = p.k;
  const int e = t.e, n0 = t.col, live = t.live;
  const int64_t m0 = t.m0;
  const int wr = wid >> 2, wc = wid & 3, c = lane & 15, qd = lane >> 4;
  const uint32_t lds0 = lds_addr(sh.data), ldsw = lds0 + kA * kABytes;
  const bool rows_role = wid >= 4;
  const int rw = wid & 3;  // among the waves of its role

  // Rows: 8 (4 rw + i) + lane / 8 in chunks of 16 bytes, the last live one in place of
  // those that are not.  Columns: 16 (kFn rw + i) + lane / 4; scales: 64 rw + lane
  // (the tile's again where it has fewer).  Columns past n repeat the last one and are
  // not stored.
  const uint8_t *src[4], *ps;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (rows_role) {
      const int row = 8 * (4 * rw + i) + (lane >> 3);
      src[i] = p.a + (m0 + min(row, live - 1)) * k * 2 + (((lane & 7) ^ x_key(row)) << 4);
    } else {
      const int col = 16 * (kFn * rw + i % kFn) + (lane >> 2);
      src[i] = p.w + ((int64_t)e * n + min(n0 + col, n - 1)) * (k / 2) +
               (((lane & 3) ^ (col >> 2 & 3)) << 4);
    }
  }
  {
    const int64_t col = (int64_t)e * n + min(n0 + (64 * rw + lane) % kBn, n - 1);
    if constexpr (kFp4) ps = p.sc + col * (k / 32);
    else ps = p.sc + col * (k / kGroup) * 2;
  }
  auto load_rows = [&](int s, uint32_t slot) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < (kPair ? 2 : 1); ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dma16_ptr(src[i] + s * (kABytes / kTileRows) + h * 128,
                  lds0 + slot + h * kHalf + (4 * rw + i) * 1024);
  };
  auto load_codes = [&](int s, uint32_t slot) __attribute__((always_inline)) {
    const uint32_t at = ldsw + slot;
#pragma unroll
    for (int i = 0; i < kFn; ++i) dma16_ptr(src[i] + s * 64, at + (kFn * rw + i) * 1024);
    // The aligned words that hold the stage's scales.
    const uint8_t* v = ps + s * (kGroup == 32 ? 8 : 4);
    if constexpr (kGroup == 128) v = (const uint8_t*)((uintptr_t)(ps + s * 2) & ~3ull);
#pragma unroll
    for (int i = 0; i < kScWords; ++i)
      dma4_ptr(v + 4 * i, at + kCodeBytes + i * 1024 + rw * 256);
  };

  // A lane reads 16 codes of its column at once, 16 qd + 0..15 of a half's 64, one
  // word for each of the half's two MFMAs, and the rows' chunks 2 qd and 2 qd + 1 to
  // match: any order along the reduction will do that both operands have.  Groups of 32
  // scaled in fp32 want an MFMA each: the upper lanes' first words and the lower lanes'
  // second ones change places, and the chunks are 0, 2, 1, 3 and 4 on.
  const int chunk = kGroup == 32 ? (qd >> 1) | (qd << 1 & 2) : 2 * qd;
  const uint32_t fx = lds0 + (wr * 64 + c) * 128 + ((chunk ^ x_key(c)) << 4);
  const uint32_t fw =
      ldsw + (wc * kFn * 16 + c) * 64 + (((qd >> 1) ^ (c >> 2)) << 4) + 8 * (qd & 1);
  const uint32_t fs = ldsw + kCodeBytes + (wc * kFn * 16 + (kFp4 ? c : 4 * qd)) * 4;
  v4f acc[kFm][kFn] = {};
  struct Frags {
    u32x4 x[2][kFm];
    uint32_t w[2][kFn];
    uint32_t s[kFp4 ? kFn : 1];
  } f[2];
  // Read u of half kOdd of a stage of codes and scales, and of its rows.
  constexpr int kReads = kFn + (kFp4 ? kFn : 0) + 2 * kFm;
  auto read = [&](Frags& r, uint32_t x_slot, uint32_t w_slot, auto parity, int u)
                  __attribute__((always_inline)) {
    constexpr int kOdd = decltype(parity)::value;
    if (u < kFn) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 v = lds_load<u32x2>(((fw + w_slot) ^ (uint32_t)(kOdd << 5)) + u * 1024);
      r.w[0][u] = v[0];
      r.w[1][u] = v[1];
      return;
    }
    u -= kFn;
    if constexpr (kFp4) {
      if (u < kFn) {
        r.s[u] = lds_load<uint32_t>(fs + w_slot + u * 64);
        return;
      }
      u -= kFn;
    }
    const int h = u / kFm, i = u % kFm;
    r.x[h][i] =
        lds_load<u32x4>(((fx + x_slot) ^ (uint32_t)(h << (kGroup == 32 ? 6 : 4))) + i * 2048);
  };
  // The scale of column 4 qd + r for half h of 64-deep stage s, in the word that
  // holds it.  Group 128: column e n + n0 + 4 qd + r starts at that times k / 128
  // scales, of which all but r k / 128 are even.
  const int per = k / BK;
  auto scale_of = [&](uint32_t v, int r, int s, int h) __attribute__((always_inline)) {
    const int up = kGroup == 32 ? h : kGroup == 64 ? s & 1 : ((r & per) ^ (s >> 1)) & 1;
    return __uint_as_float(up ? v & 0xffff0000u : v << 16);
  };
  auto mfma = [](const bf16x8& w, const u32x4& x, const v4f& d) __attribute__((always_inline)) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, x), d, 0, 0, 0);
  };
  // The products of half kOdd of a stage, from registers; next(u) is called between
  // them, u = 0 .. kReads - 1.  The order is fixed (sched_fence): left to itself the compiler
  // puts the reads first and waits for them.
  auto compute = [&](Frags& r, int s, uint32_t slot, auto parity, auto&& next)
                     __attribute__((always_inline)) {
    constexpr int kOdd = decltype(parity)::value;
    int u = 0;
    auto between = [&]() __attribute__((always_inline)) {
      sched_fence();
      if (u < kReads) next(u);
      ++u;
      sched_fence();
    };
    if constexpr (kFp4) {
      auto values = [&](int g) __attribute__((always_inline)) {  // column tile g / 2, half g % 2
        const int j = g >> 1, h = g & 1;
        // The lane's 16 codes are of one group: byte qd / 2 of the half's two.
        const uint32_t scale = r.s[j] >> (16 * kOdd + 8 * (qd >> 1)) & 0xffu;
        return fp4_values(r.w[h][j], __uint_as_float(scale << 23));
      };
      bf16x8 v = values(0), after;
#pragma unroll
      for (int g = 0; g < 2 * kFn; ++g) {
#pragma unroll
        for (int i = 0; i < kFm; ++i) {
          acc[i][g >> 1] = mfma(v, r.x[g & 1][i], acc[i][g >> 1]);
          if (i == 1 && g + 1 < 2 * kFn) after = values(g + 1);
          between();
        }
        v = after;
      }
    } else {
      const bf16x8 c8 = __builtin_bit_cast(bf16x8, u32x4{kMinus8, kMinus8, kMinus8, kMinus8});
      constexpr int kParts = kGroup == 32 ? 2 : 1;  // groups of a half, at most a half long
      if constexpr (kGroup == 32) {
#pragma unroll
        for (int j = 0; j < kFn; ++j) {
          const auto w = __builtin_amdgcn_permlane32_swap(r.w[0][j], r.w[1][j], false, false);
          r.w[0][j] = w[0];
          r.w[1][j] = w[1];
        }
      }
      v4f off[kParts][kFm];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kFm; ++i) {
          const v4f zero = {0.f, 0.f, 0.f, 0.f};
          off[h % kParts][i] = mfma(c8, r.x[h][i], h < kParts ? zero : off[0][i]);
          between();
        }
      // Scales of the lane's 4 columns in tile j.
      auto scales = [&](int j) __attribute__((always_inline)) {
        return lds_load<u32x4>(fs + slot + (kScWords == 2 ? kOdd * 1024 : 0) + j * 64);
      };
      auto add_row = [&](int j, int i, int h, const u32x4& sw, const v4f& part)
                         __attribute__((always_inline)) {
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) acc[i][j][c4] += part[c4] * scale_of(sw[c4], c4, s, h);
      };
      bf16x8 v = int4_values(r.w[0][0]), after;
      if constexpr (kParts == 1) {
        // A tile's group is complete with its second MFMAs; it is scaled between the
        // next tile's, when they are done.
        v4f part[kFn][kFm];
        u32x4 sw[kFn];
#pragma unroll
        for (int j = 0; j < kFn; ++j) sw[j] = scales(j);
#pragma unroll
        for (int g = 0; g < 2 * kFn; ++g) {
          const int h = g / kFn, j = g % kFn;
#pragma unroll
          for (int i = 0; i < kFm; ++i) {
            part[j][i] = mfma(v, r.x[h][i], h ? part[j][i] : off[0][i]);
            if (i == 1 && g + 1 < 2 * kFn) after = int4_values(r.w[(g + 1) / kFn][(g + 1) % kFn]);
            if (h && j > 0) add_row(j - 1, i, h, sw[j - 1], part[j - 1][i]);
            between();
          }
          v = after;
        }
#pragma unroll
        for (int i = 0; i < kFm; ++i) add_row(kFn - 1, i, 1, sw[kFn - 1], part[kFn - 1][i]);
      } else {
#pragma unroll
        for (int j = 0; j < kFn; ++j) {
          const u32x4 sw = scales(j);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v4f part[kFm];
#pragma unroll
            for (int i = 0; i < kFm; ++i) {
              part[i] = mfma(v, r.x[h][i], off[h][i]);
              if (i == 1 && 2 * j + h + 1 < 2 * kFn)
                after = int4_values(r.w[(h + 1) & 1][j + (h + 1) / 2]);
              between();
            }
            v = after;
#pragma unroll
            for (int i = 0; i < kFm; ++i) add_row(j, i, h, sw, part[i]);
          }
        }
      }
    }
    while (u < kReads) between();
  };

  const int stages = k / 128, steps = 2 * stages, a_stages = kPair ? stages : steps;
  wait_vmcnt<0>();  // the last item's stores do not enter the counts below
  if (rows_role) {
    for (int s = 0; s < kA && s < a_stages; ++s) load_rows(s, s * kABytes);
    wait_ahead<kALoads, kA - 1>(min(kA - 1, a_stages - 1));
  } else {
    for (int s = 0; s < kW - 1 && s < stages; ++s) load_codes(s, s * kWBytes);
    wait_ahead<kWLoads, kW - 2>(min(kW - 2, stages - 1));
  }
  barrier();
#pragma unroll
  for (int u = 0; u < kReads; ++u) read(f[0], 0, 0, std::integral_constant<int, 0>(), u);
  // Slots: of the rows computed (loaded anew once they are in registers), and of the
  // codes computed (int4's scales are still read there) and before them.
  uint32_t x_now = 0, w_now = 0, w_old = (kW - 1) * kWBytes;
  auto bump = [](uint32_t at, uint32_t by, uint32_t end) __attribute__((always_inline)) {
    return at + by == end ? 0 : at + by;
  };
  // Half s of the reduction.  Before the next half's fragments are read, it has landed
  // for all waves, and all have read the slots that are then loaded anew: the rows' of
  // this half's stage, and the codes' of the stage before (they are loaded every second
  // half, kW - 1 stages ahead).  A pair's second half is there with its first.
  auto step = [&](int s, auto parity) __attribute__((always_inline)) {
    constexpr int kOdd = decltype(parity)::value;
    constexpr bool kSync = !kPair || kOdd, kCodes = kPair ? kOdd : !kOdd;
    const int t2 = s >> 1, as = kPair ? t2 : s;
    const uint32_t x_next = kSync ? bump(x_now, kABytes, kA * kABytes) : x_now;
    const uint32_t w_next = kOdd ? bump(w_now, kWBytes, kW * kWBytes) : w_now;
    if constexpr (kSync) {
      constexpr int kAhead = kPair ? kW - 3 : kW - 2;
      if (rows_role) wait_ahead<kALoads, kA - 2>(min(kA - 2, a_stages - 2 - as));
      else if (kOdd) wait_ahead<kWLoads, kAhead>(min(kAhead, stages - 2 - t2));
      wait_lgkm0();
      barrier();
      if (rows_role) {
        if (as + kA < a_stages) load_rows(as + kA, x_now);
      } else if (kCodes) {
        if (t2 + kW - 1 < stages) load_codes(t2 + kW - 1, w_old);
      }
    }
    // (After the last step the fragments read are not used.)
    compute(f[kOdd], s, w_now, parity, [&](int u) __attribute__((always_inline)) {
      read(f[kOdd ^ 1], x_next + (kPair && !kOdd ? kHalf : 0), w_next,
           std::integral_constant<int, kOdd ^ 1>(), u);
    });
    if (kOdd) {
      w_old = w_now;
      w_now = w_next;
    }
    x_now = x_next;
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, std::integral_constant<int, 0>());
    step(s + 1, std::integral_constant<int, 1>());
  }
  // The last stages have been read (int4's scales are asked for after the steps' waits).
  wait_lgkm0();
  barrier();

  // The lane holds columns 4 qd + 0..3 of tile j for row c of tile i; two lane
  // swaps make 8 neighbouring columns of two tiles: 16-byte stores.
  const int tc = n0 + wc * kFn * 16 + (lane >> 5) * 16 + (lane >> 4 & 1) * 8;
#pragma unroll
  for (int i = 0; i < kFm; ++i) {
    const int m = wr * 64 + i * 16 + c;
    uint16_t* row = p.out + (m0 + m) * n + tc;
#pragma unroll
    for (int j = 0; j < kFn; j += 2) {
      const u32x4 o = pack_tiles(acc[i][j], acc[i][j + 1]);
      if (m < live && tc + j * 16 < n) *reinterpret_cast<u32x4*>(row + j * 16) = o;
    }
  }
}

// ------------------------------------------------------------------- tall

// MXFP4, 256 rows, 256 columns: eight waves, 2 by 4, of 128 x 64.  A code is decoded for
// twice as many rows and LDS is read a tenth less than with 128 rows (8192 rows, 8 x 4096
// x 7168: 462 -> 418 us; 6500 rows, 16 x 4096 x 4096: 242 -> 211).  128 sums to a
// thread leave room for one set of row fragments, 32 deep: each is read anew as soon as
// its last product has been issued.  Roles and stages as in wide; 3 stages of rows, 2 of
// codes.
__device__ __forceinline__ void tall(Shared& sh, const Args& p, const Item& t, int lane,
                                     int wid) {
  constexpr int kFm = 8, kFn = 4, kBn = 64 * kFn;
  constexpr int kA = 3, kW = 2;                                    // stages in LDS
  constexpr int kABytes = kTallRows * 128, kCodeBytes = kBn * 64, kWBytes = kCodeBytes + 1024;
  static_assert(kA * kABytes + kW * kWBytes <= kDataBytes);
  const int n = p.n, k = p.k;
  const int e = t.e, n0 = t.col, live = t.live;
  const int64_t m0 = t.m0;
  const int wr = wid >> 2, wc = wid & 3, c = lane & 15, qd = lane >> 4;
  const uint32_t lds0 = lds_addr(sh.data), ldsw = lds0 + kA * kABytes;
  const bool rows_role = wid >= 4;
  const int rw = wid & 3;

  // As in wide: rows 8 (8 rw + i) + lane / 8, columns 16 (4 rw + i) + lane / 4.  Their
  // offsets (256 lines of less than 2^16 bytes) are formed anew each time: held, they
  // would not leave room for the sums.
  const int64_t col0 = (int64_t)e * n + n0;
  const uint8_t* const base = rows_role ? p.a + m0 * k * 2 : p.w + col0 * (k / 2);
  const uint8_t* const base_sc = p.sc + col0 * (k / 32);
  const uint32_t last = rows_role ? live - 1 : n - 1 - n0, pitch = rows_role ? k * 2 : k / 2;
  auto load_rows = [&](int s, uint32_t slot) __attribute__((always_inline)) {
    const uint8_t* from = settled(base + s * 128);
    const uint32_t l = lane_now();
    const uint32_t swz = ((l & 7) ^ x_key(l >> 3)) << 4;
#pragma unroll
    for (int i = 0; i < kFm; ++i) {
      const uint32_t row = min((uint32_t)(8 * (kFm * rw + i)) + (l >> 3), last);
      dma16(from, __umul24(row, pitch) + (swz ^ (uint32_t)((i & 1) << 6)),
            lds0 + slot + (kFm * rw + i) * 1024);
      sched_fence();
    }
  };
  auto load_codes = [&](int s, uint32_t slot) __attribute__((always_inline)) {
    const uint32_t at = ldsw + slot;
    const uint8_t* from = settled(base + s * 64);
    const uint32_t l = lane_now();
    const uint32_t swz = ((l & 3) ^ (l >> 4)) << 4;
#pragma unroll
    for (int i = 0; i < kFn; ++i) {
      const uint32_t col = min((uint32_t)(16 * (kFn * rw + i)) + (l >> 2), last);
      dma16(from, __umul24(col, pitch) + swz, at + (kFn * rw + i) * 1024);
      sched_fence();
    }
    dma4(base_sc + s * 4, __umul24(min(64 * rw + l, last), (uint32_t)(k / 32)),
         at + kCodeBytes + rw * 256);
  };

  const uint32_t fx = lds0 + (wr * 128 + c) * 128 + (((2 * qd) ^ x_key(c)) << 4);
  const uint32_t fw =
      ldsw + (wc * kFn * 16 + c) * 64 + (((qd >> 1) ^ (c >> 2)) << 4) + 8 * (qd & 1);
  const uint32_t fs = ldsw + kCodeBytes + (wc * kFn * 16 + c) * 4;
  v4f acc[kFm][kFn] = {};
  u32x4 x[kFm];
  uint32_t w[2][kFn], sc[kFn];
  bf16x8 v;
  auto read_x = [&](uint32_t slot, int h, int i) __attribute__((always_inline)) {
    x[i] = lds_load<u32x4>(((fx + slot) ^ (uint32_t)(h << 4)) + i * 2048);
  };
  auto read_w = [&](uint32_t slot, int odd, int j) __attribute__((always_inline)) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 d = lds_load<u32x2>(((fw + slot) ^ (uint32_t)(odd << 5)) + j * 1024);
    w[0][j] = d[0];
    w[1][j] = d[1];
  };
  auto values = [&](int j, int h, int odd) __attribute__((always_inline)) {
    const uint32_t scale = sc[j] >> (16 * odd + 8 * (qd >> 1)) & 0xffu;
    return fp4_values(w[h][j], __uint_as_float(scale << 23));
  };
  // Column tile j with 32 of the reduction; the next one's values are made at row d, and
  // between(i) is called after row i's product.
  auto products = [&](int j, int d, auto&& next, auto&& between) __attribute__((always_inline)) {
    bf16x8 after = v;
#pragma unroll
    for (int i = 0; i < kFm; ++i) {
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, x[i]),
                                                          acc[i][j], 0, 0, 0);
      if (i == d) after = next();
      sched_fence();
      between(i);
      sched_fence();
    }
    v = after;
  };

  const int stages = k / 128, steps = 2 * stages;
  wait_vmcnt<0>();  // the last item's stores do not enter the counts below
  if (rows_role) {
    for (int s = 0; s < kA && s < steps; ++s) load_rows(s, s * kABytes);
    wait_ahead<kFm, kA - 1>(min(kA - 1, steps - 1));
  } else {
    for (int s = 0; s < kW && s < stages; ++s) load_codes(s, s * kWBytes);
    wait_ahead<kFn + 1, kW - 1>(min(kW - 1, stages - 1));
  }
  barrier();
#pragma unroll
  for (int j = 0; j < kFn; ++j) {
    read_w(0, 0, j);
    sc[j] = lds_load<uint32_t>(fs + j * 64);
  }
#pragma unroll
  for (int i = 0; i < kFm; ++i) read_x(0, 0, i);
  v = values(0, 0, 0);
  uint32_t x_now = 0, w_now = 0;
  auto nothing = [](int) __attribute__((always_inline)) {};
  // Half s of a stage of codes.  Once its rows are in registers for all waves and the
  // next half has landed, their slot is loaded anew, and that of the codes' stage, whose
  // last ones were read a half before.
  auto step = [&](int s, auto parity) __attribute__((always_inline)) {
    constexpr int kOdd = decltype(parity)::value;
    const uint32_t x_next = x_now + kABytes == kA * kABytes ? 0 : x_now + kABytes;
    const uint32_t w_next = kOdd ? (w_now ? 0 : kWBytes) : w_now;
    products(0, 2, [&]() { return values(1, 0, kOdd); }, nothing);
    products(1, 2, [&]() { return values(2, 0, kOdd); }, nothing);
    products(2, 2, [&]() { return values(3, 0, kOdd); }, nothing);
    products(3, 2, [&]() { return values(0, 1, kOdd); }, [&](int i) { read_x(x_now, 1, i); });
    products(0, 2, [&]() { return values(1, 1, kOdd); }, nothing);
    products(1, 2, [&]() { return values(2, 1, kOdd); }, nothing);
    products(2, 2, [&]() { return values(3, 1, kOdd); }, nothing);
    int role = wid;
    asm volatile("" : "+s"(role));  // compared here: a held comparison takes a vector register
    const bool rows_now = role >= 4;
    if (rows_now) wait_ahead<kFm, 1>(min(1, steps - 2 - s));
    else if (kOdd) wait_vmcnt<0>();
    wait_lgkm0();
    barrier();
    if (rows_now) {
      if (s + kA < steps) load_rows(s + kA, x_now);
    } else if (kOdd) {
      if ((s >> 1) + kW < stages) load_codes((s >> 1) + kW, w_now);
    }
    uint32_t fs_next = fs + w_next;
    asm volatile("" : "+v"(fs_next));  // one address
    // (After the last half what is read is not used.)
    products(3, 7, [&]() { return values(0, 0, kOdd ^ 1); }, [&](int i) {
      if (i < kFn) {
        read_w(w_next, kOdd ^ 1, i);
        if (kOdd) sc[i] = lds_load<uint32_t>(fs_next + i * 64);
      }
      read_x(x_next, 0, i);
    });
    x_now = x_next;
    w_now = w_next;
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, std::integral_constant<int, 0>());
    step(s + 1, std::integral_constant<int, 1>());
  }
  wait_lgkm0();
  barrier();  // the last stages have been read

  const int l = lane_now(), row0 = wr * 128 + (l & 15);
  const int tc = n0 + wc * kFn * 16 + (l >> 5) * 16 + (l >> 4 & 1) * 8;
#pragma unroll
  for (int i = 0; i < kFm; ++i) {
    const int m = row0 + i * 16;
    uint16_t* row = p.out + (m0 + m) * n + tc;
#pragma unroll
    for (int j = 0; j < kFn; j += 2) {
      const u32x4 o = pack_tiles(acc[i][j], acc[i][j + 1]);
      if (m < live && tc + j * 16 < n) *reinterpret_cast<u32x4*>(row + j * 16) = o;
    }
  }
}

template <int kGroup>
__global__ __launch_bounds__(kThreads) void w4_kernel(
    const uint8_t* __restrict__ a, const uint8_t* __restrict__ w, const uint8_t* __restrict__ sc,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ status, int64_t capacity, int n,
    int k, int E, int align, uint16_t* __restrict__ out) {
  __shared__ Shared sh;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Bytes of 64 columns' scales, and the room for an item's (of 128, at least).
  const int sc64 = kNarrowCols * (k / BK) * Scales<kGroup>::kBytes;
  constexpr int kRoom = (kDataBytes - kPartBytes) / 2 / 1024 * 1024;
  const Args p = {a, w, sc, min((int64_t)__builtin_amdgcn_readfirstlane(status[0]), capacity), n, k, E, align, out,
                  2 * sc64 <= kRoom};
  for (int e = threadIdx.x; e < E; e += kThreads) sh.pe[e] = psum[e];
  __syncthreads();
  if (wid == 0) list_items<kGroup>(sh, p, lane);
  __syncthreads();
  const int groups = __builtin_amdgcn_readfirstlane(sh.gp[kWide][E]);
  // 256 columns where that makes a round of items or more, and 256 rows, too.
  const int NT256 = (n + 255) / 256, NT128 = n / 128;
  const int shape = __builtin_amdgcn_readfirstlane(
      kGroup != 0 ? 0 : sh.tile == kTallRows ? 2 : (uint32_t)groups * (uint32_t)NT256 >= gridDim.x);
  const int NTW = shape ? NT256 : NT128;
  // A last round that leaves half of the workgroups idle takes its tiles in halves, and
  // tall ones of a quarter of them in quarters (128-row tiles of 256 columns, 8192 rows,
  // 8 x 4096 x 7168, about 68 row groups of 16 tiles: 490 -> 467 us; 4000 rows, 8 x 2048 x 2048:
  // 63 -> 52).
  uint32_t nwide = (uint32_t)groups * (uint32_t)NTW, whole = nwide;
  int split = 0;  // log2 of the parts
  const uint32_t rest = nwide % gridDim.x;
  if (shape && rest * 2 <= gridDim.x) split = shape == 2 && rest * 4 <= gridDim.x ? 2 : 1;
  if (split) {
    whole -= rest;
    nwide = whole + (rest << split);
  }
  const int two = __builtin_amdgcn_readfirstlane(sh.gp[kTwo][E]);
  const int one = __builtin_amdgcn_readfirstlane(sh.gp[kOne][E]);
  // Groups of columns in a narrow item: 1, 2, 4 or 8, whichever takes least by
  // blocks of 64 columns in a workgroup's rounds, and about six of them for each item's
  // join.
  auto groups_of = [&](int entries, int cols) __attribute__((always_inline)) {
    int cs = 1;
    uint32_t least = 0xffffffffu;
    for (int i = 1; i <= kWaves; i *= 2) {
      if (n % (cols * i) || (int64_t)(sc64 / kNarrowCols) * cols * i > kRoom) break;
      const uint32_t items = (uint32_t)entries * (uint32_t)(n / (cols * i));
      const uint32_t cost =
          (items + gridDim.x - 1) / gridDim.x * (uint32_t)(i * (cols / kNarrowCols) * (k / BK) + 6);
      if (cost < least) least = cost, cs = i;
    }
    return cs;
  };
  constexpr int kTiles2 = 8, kTiles1 = 4;
  const int cs2 = groups_of(two, 16 * kTiles2), cs1 = groups_of(one, 16 * kTiles1);
  const uint32_t end2 = nwide + (uint32_t)two * (uint32_t)(n / (16 * kTiles2 * cs2));
  const uint32_t nitems = end2 + (uint32_t)one * (uint32_t)(n / (16 * kTiles1 * cs1));
  uint32_t base = 0;
  for (;; base += gridDim.x) {
    const uint32_t item = round_item(base, nitems);
    if (item >= nwide) break;
    const bool part = item >= whole;
    const uint32_t of = item - whole;
    Item t = uniform(decode(sh, p, kWide, part ? whole + (of >> split) : item, NTW,
                            shape ? 256 : 128, shape == 2 ? kTallRows : kTileRows));
    int now = shape;
    if (part) {
      // Tall ones go in halves of 128 rows or in quarters, others in halves of 128 columns.
      const int cols = split - shape / 2, rows = shape / 2;  // log2 of parts either way
      t.col += (int)of % (1 << cols) * 128;
      const int down = (int)(of >> cols) % (1 << rows) * 128;
      t.m0 += down;
      t.live = min(t.live - down, rows ? 128 : t.live);
      now -= cols + rows;
      if (t.col >= n || t.live <= 0) continue;
    }
    int w = wid;
    now = __builtin_amdgcn_readfirstlane(now);
    Args q = p;
    asm volatile("" : "+s"(w), "+s"(now), "+s"(q.n), "+s"(q.k));
    if (now == 2) {
      if constexpr (kGroup == 0) tall(sh, q, t, lane_now(), w);
    } else if (now == 1) {
      if constexpr (kGroup == 0) wide<kGroup, 4>(sh, q, t, lane_now(), w);
    } else {
      wide<kGroup, 2>(sh, q, t, lane_now(), w);
    }
  }
  narrow<kGroup, 2, kTiles2>(sh, p, nwide, end2, nitems, cs2, base, lane_now(), wid);
  narrow<kGroup, 1, kTiles1>(sh, p, end2, nitems, nitems, cs1, base, lane_now(), wid);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_grouped_gemm_w4(const void* a, const void* w, const void* w_scale,
                                          moe_w4_fmt fmt, int group, const int32_t* psum,
                                          const int32_t* status, int64_t capacity, int n, int k,
                                          int num_experts, int align, void* out, void* stream) {
  if (capacity < 0 || capacity > (1LL << 30) || n <= 0 || k <= 0 || n % 128 || k % BK ||
      num_experts < 1 || num_experts > MOE_MAX_EXPERTS)
    return MOE_ERR_SHAPE;
  if (align < MOE_MIN_ALIGN || align > MOE_MAX_ALIGN || (align & (align - 1)))
    return MOE_ERR_UNSUPPORTED;
  if (capacity % align != 0) return MOE_ERR_SHAPE;
  if (fmt == MOE_W4_INT4 ? group != 32 && group != 64 && group != 128
                         : fmt != MOE_W4_MXFP4 || group != 32)
    return MOE_ERR_UNSUPPORTED;
  if (n / 64 > kMaxBlocks64 || k / 64 > kMaxBlocks64) return MOE_ERR_UNSUPPORTED;
  if (!psum || !status || !w || !w_scale) return MOE_ERR_NULL;
  if (capacity > 0 && (!a || !out)) return MOE_ERR_NULL;
  if ((uintptr_t)a % 16 || (uintptr_t)w % 16 || (uintptr_t)out % 16 || (uintptr_t)w_scale % 16)
    return MOE_ERR_ALIGNMENT;
  if (capacity == 0) return MOE_OK;
  const int64_t bytes = capacity * n * 2, cols = (int64_t)num_experts * n;
  if (overlap(out, bytes, a, capacity * k * 2) || overlap(out, bytes, w, cols * (k / 2)) ||
      overlap(out, bytes, w_scale, cols * (k / group) * (fmt == MOE_W4_INT4 ? 2 : 1)) ||
      overlap(out, bytes, psum, num_experts * 4LL) || overlap(out, bytes, status, 8))
    return MOE_ERR_UNSUPPORTED;
  // A workgroup per CU (its LDS) walks the items of the device's layout.
  int64_t grid = ((capacity + kNarrowRows - 1) / kNarrowRows + num_experts) *
                 (int64_t)(n / kNarrowCols);
  if (grid > device_cus()) grid = device_cus();
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  auto kern = fmt == MOE_W4_MXFP4 ? w4_kernel<0>
              : group == 32       ? w4_kernel<32>
              : group == 64       ? w4_kernel<64>
                                  : w4_kernel<128>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), (const uint8_t*)a, (const uint8_t*)w,
                     (const uint8_t*)w_scale, psum, status, capacity, n, k, num_experts, align,
                     (uint16_t*)out);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
