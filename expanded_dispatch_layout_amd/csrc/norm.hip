// moe_layer_norm, moe_layer_norm_backward: the norm of the residual stream in
// front of an MoE layer, with the branch added on the way, and its gradient.
//
//   h = x + branch,  y = (h - mu) r w + b,  r = 1 / sqrt(mean((h - mu)^2) + eps)
//   (RMS: mu = 0)
//   g = (dy + dy2) w,  xh = (h - mu) r
//   dh = r (g - mean(g) - xh mean(g xh)) + dsum   (RMS: without mean(g))
//   dw = sum over rows of (dy + dy2) xh,  db = sum over rows of dy + dy2
//
// HBM-bound: every value is read and written once; a row stays in registers
// between its sums and its outputs.  The variance is summed about the mean
// (a second pass over the registers), so a mean that is large against the
// deviation costs no digits.
// Forward: a wave or a workgroup per row, by its length.  16384 rows of 6144, fp32
// stream with a branch: 245 us, 4.9 TB/s, the rate of a plain copy (accesses past the
// caches: 254 to 262).  Backward: 16384 rows of 7168 in bf16, two gradients and the
// stream's: 211 us, 5.6 TB/s, of which 7.4 join the weight's gradient.
#include <initializer_list>

#include "lds_dma.hpp"

namespace moe {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kMaxHidden = 8192;

// 8 consecutive values of a bf16 or fp32 array as floats, and back.
template <bool kF32>
struct Chunk;
template <>
struct Chunk<false> {
  u32x4 v;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    v = *reinterpret_cast<const u32x4*>((const uint16_t*)p + at);
  }
  __device__ __forceinline__ void load_once(const void* p, int64_t at) {  // past the caches
    v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const uint16_t*)p + at));
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
  }
};
template <>
struct Chunk<true> {
  v4f lo, hi;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    lo = *reinterpret_cast<const v4f*>((const float*)p + at);
    hi = *reinterpret_cast<const v4f*>((const float*)p + at + 4);
  }
  __device__ __forceinline__ void load_once(const void* p, int64_t at) {
    lo = __builtin_nontemporal_load(reinterpret_cast<const v4f*>((const float*)p + at));
    hi = __builtin_nontemporal_load(reinterpret_cast<const v4f*>((const float*)p + at + 4));
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? lo[i] : hi[i - 4]; }
};

template <bool kF32>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (kF32) {
    *reinterpret_cast<v4f*>((float*)p + at) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f*>((float*)p + at + 4) = v4f{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4*>((uint16_t*)p + at) =
        u32x4{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7])};
  }
}

// The same in bf16, past the caches.
__device__ __forceinline__ void store8_once(void* p, int64_t at, const float (&v)[8]) {
  __builtin_nontemporal_store(
      u32x4{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7])},
      reinterpret_cast<u32x4*>((uint16_t*)p + at));
}

// A gain or bias vector, bf16 or fp32 (the same for every row: from the caches).
__device__ __forceinline__ void load_gain(const void* p, bool f32, int at, float (&v)[8]) {
  if (f32) {
    Chunk<true> c;
    c.load(p, at);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c.get(i);
  } else {
    Chunk<false> c;
    c.load(p, at);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c.get(i);
  }
}

constexpr int kThreads = 256, kWaves = kThreads / kWave;

// kTeam waves share a row (1, or all of the workgroup); a thread holds kCh
// chunks of 8 columns.
template <bool kF32, int kTeam, int kCh>
__global__ __launch_bounds__(kThreads) void norm_kernel(
    const void* x, int64_t x_stride, const uint16_t* __restrict__ branch,
    const void* __restrict__ weight, const void* __restrict__ bias, bool w_f32, bool rms,
    float eps, const int32_t* __restrict__ psum_rank, int nsrc, int64_t rows, int hidden,
    void* sum, uint16_t* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float part[2][kWaves];
  const int wid = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = kTeam == 1 ? lane : threadIdx.x;
  constexpr int kRows = kWaves / kTeam, kStep = kTeam * kWave * 8;
  const int64_t nv = valid_rows(psum_rank, nsrc, rows);
  const float inv = 1.0f / (float)hidden;
  int slot = 0;
  auto team_sum = [&](float v) __attribute__((always_inline)) {
    v = wave_sum_f(v);
    if constexpr (kTeam > 1) {
      if (lane == 0) part[slot][wid] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) v += part[slot][i];
      slot ^= 1;  // the next sum goes elsewhere: one barrier each
    }
    return v;
  };
  for (int64_t r = (int64_t)blockIdx.x * kRows + (kTeam == 1 ? wid : 0); r < nv;
       r += (int64_t)gridDim.x * kRows) {
    float h[kCh][8];
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
      const int at = t * 8 + c * kStep;
      if (at < hidden) {
        Chunk<kF32> a;
        a.load(x, r * x_stride + at);
        Chunk<false> b;
        if (branch) b.load(branch, r * hidden + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[c][i] = a.get(i);
          if (branch) {
            h[c][i] += b.get(i);
            // The norm is of the stream as it is kept, which the backward
            // pass reads again: rounded to its type.
            if constexpr (!kF32) h[c][i] = bf16_to_f32(f32_to_bf16_rne(h[c][i]));
          }
        }
        if (sum) store8<kF32>(sum, r * hidden + at, h[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += h[c][i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = 0.f;
      }
    }
    const float mu = rms ? 0.f : team_sum(s) * inv;
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < kCh; ++c)
      if (t * 8 + c * kStep < hidden) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[c][i] -= mu;
          q += h[c][i] * h[c][i];
        }
      }
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(team_sum(q) * inv + eps));
    if (t == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
      const int at = t * 8 + c * kStep;
      if (at >= hidden) continue;
      float w[8], b[8], o[8];
      load_gain(weight, w_f32, at, w);
      if (bias) load_gain(bias, w_f32, at, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = h[c][i] * rs * w[i];
        if (bias) o[i] += b[i];
      }
      store8<false>(y, r * hidden + at, o);
    }
  }
}

// ------------------------------------------------------------ backward

constexpr int kBackThreads = 512, kBackWaves = kBackThreads / kWave;
// bf16 dx beyond this goes past the caches: nothing of it would be left for its reader
// (16384 rows of 7168, two gradients and the stream's: 227 us with plain stores, 210 so;
// 12288 rows, one gradient: 106 and 98).  fp32 gains nothing for sure (16384 rows of 7168:
// 347 and 344; of 6144, one gradient: 194 and 201; 32768 of 2048: 204 and 197).
constexpr int64_t kCached = 128 << 20;
constexpr int kParts = 256;  // workgroups, and partial sums of the weight's gradient

// kTeam waves share a row, kU rows at a time; a thread holds kCh chunks of 8
// columns, and over all its rows the sums of its columns' dw and db.  The next rows
// are asked for before the present ones are worked on (16384 rows of 7168, plain stores:
// 246 us without, 227 so; two rows at a time spill at this width: 519).  The workgroup's
// sums go to its own place in the workspace (512 workgroups in place of 256: 247).
// Loads are not conditional, so that the compiler can count them: columns and rows past
// the end repeat the last ones, with a gradient of 0.  (Where those hold a NaN, the sums
// have one already.)
template <bool kF32, bool kTwo, bool kSum, int kTeam, int kCh, int kU>
__global__ __launch_bounds__(kBackThreads) void norm_backward_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ dy2, const void* __restrict__ x,
    int64_t x_stride, const void* __restrict__ weight, bool w_f32, bool rms,
    const float* __restrict__ mean, const float* __restrict__ rstd, const void* dsum,
    const int32_t* __restrict__ psum_rank, int nsrc, int64_t rows, int hidden, bool once,
    void* dx, float* __restrict__ parts) {
  constexpr int kTeams = kBackWaves / kTeam, kStep = kTeam * kWave * 8;
  __shared__ float part[2][kBackWaves][2 * kU];
  __shared__ float join[kTeams > 1 ? kBackThreads * 8 : 1];
  const int wid = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int team = wid / kTeam, t = threadIdx.x % (kTeam * kWave);
  const int64_t nv = valid_rows(psum_rank, nsrc, rows);
  const float inv = 1.0f / (float)hidden;
  const float* mean_or = rms ? rstd : mean;  // (RMS: read and not used)
  int at[kCh];
  bool ok[kCh];
  float w[kCh][8], dw[kCh][8] = {}, db[kCh][8] = {};
#pragma unroll
  for (int c = 0; c < kCh; ++c) {
    ok[c] = t * 8 + c * kStep < hidden;
    at[c] = ok[c] ? t * 8 + c * kStep : hidden - 8;
    load_gain(weight, w_f32, at[c], w[c]);
  }
  struct Rows {
    Chunk<false> a[kU][kCh], a2[kU][kCh];
    Chunk<kF32> x[kU][kCh], ds[kU][kCh];
    float mu[kU], rs[kU];
  } set[2];
  const int64_t stride = (int64_t)gridDim.x * (kTeams * kU);
  const int64_t first = ((int64_t)blockIdx.x * kTeams + team) * kU;
  const int64_t block0 = (int64_t)blockIdx.x * (kTeams * kU);
  const int rounds = block0 < nv ? (int)((nv - block0 + stride - 1) / stride) : 0;
  auto load = [&](Rows& s, int round) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t r = min(first + round * stride + u, nv - 1);
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        s.a[u][c].load_once(dy, r * hidden + at[c]);
        if constexpr (kTwo) s.a2[u][c].load_once(dy2, r * hidden + at[c]);
        s.x[u][c].load_once(x, r * x_stride + at[c]);
        if constexpr (kSum) s.ds[u][c].load_once(dsum, r * hidden + at[c]);
      }
      s.mu[u] = mean_or[r];
      s.rs[u] = rstd[r];
    }
  };
  auto grad = [&](const Rows& s, int u, int c, int i, bool live) __attribute__((always_inline)) {
    float d = s.a[u][c].get(i);
    if constexpr (kTwo) d += s.a2[u][c].get(i);
    return live && ok[c] ? d : 0.f;
  };
  int slot = 0;
  auto work = [&](const Rows& s, int round) __attribute__((always_inline)) {
    float s1[kU], s2[kU], mu[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const bool live = first + round * stride + u < nv;
      mu[u] = rms ? 0.f : s.mu[u];
      s1[u] = s2[u] = 0.f;
#pragma unroll
      for (int c = 0; c < kCh; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = grad(s, u, c, i, live);
          const float xh = (s.x[u][c].get(i) - mu[u]) * s.rs[u];
          dw[c][i] += d * xh;
          db[c][i] += d;
          s1[u] += d * w[c][i];
          s2[u] += d * w[c][i] * xh;
        }
      s1[u] = wave_sum_f(s1[u]);
      s2[u] = wave_sum_f(s2[u]);
      if constexpr (kTeam > 1) {
        if (lane == 0) {
          part[slot][wid][2 * u] = s1[u];
          part[slot][wid][2 * u + 1] = s2[u];
        }
      }
    }
    if constexpr (kTeam > 1) {
      wait_lgkm0();
      barrier();
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        s1[u] = s2[u] = 0.f;
#pragma unroll
        for (int i = 0; i < kTeam; ++i) {
          s1[u] += part[slot][team * kTeam + i][2 * u];
          s2[u] += part[slot][team * kTeam + i][2 * u + 1];
        }
      }
      slot ^= 1;  // the next rows' sums go elsewhere: one barrier per round
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t r = first + round * stride + u;
      if (r >= nv) continue;
      const float m1 = rms ? 0.f : s1[u] * inv, m2 = s2[u] * inv;
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = grad(s, u, c, i, true);
          const float xh = (s.x[u][c].get(i) - mu[u]) * s.rs[u];
          o[i] = s.rs[u] * (d * w[c][i] - m1 - xh * m2);
          if constexpr (kSum) o[i] += s.ds[u][c].get(i);
        }
        if (ok[c]) {
          if (!kF32 && once) {
            // (Set apart: the compiler joins the two branches otherwise, as plain stores.)
            asm volatile("; past the caches");
            store8_once(dx, r * hidden + at[c], o);
            asm volatile("; past the caches");
          } else {
            store8<kF32>(dx, r * hidden + at[c], o);
          }
        }
      }
    }
  };
  if (rounds > 0) load(set[0], 0);
  for (int i = 0; i < rounds; i += 2) {  // (a round past the last has no live row)
    load(set[1], i + 1);
    work(set[0], i);
    load(set[0], i + 2);
    work(set[1], i + 1);
  }
  if (!parts) return;
  // [workgroup][dw, db][hidden]; the teams of a workgroup are summed in order.
  float* out = parts + (int64_t)blockIdx.x * 2 * hidden;
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = which ? db[c][i] : dw[c][i];
      if constexpr (kTeams > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) join[threadIdx.x * 8 + i] = v[i];
        __syncthreads();
        if (team == 0) {
          for (int k = 1; k < kTeams; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += join[(k * kTeam * kWave + t) * 8 + i];
        }
      }
      if (team == 0 && ok[c]) store8<true>(out, (int64_t)which * hidden + at[c], v);
    }
}

// Sum of the workgroups' parts, 64 columns to a workgroup of 16 threads of 4
// columns by 16 parts, in a fixed order.
__global__ __launch_bounds__(256) void norm_join_kernel(const float* __restrict__ parts,
                                                        int nparts, int hidden, void* dweight,
                                                        void* dbias, bool f32, bool accumulate) {
  __shared__ v4f join[256];
  const int which = blockIdx.y;
  const int col = blockIdx.x * 64 + (threadIdx.x & 15) * 4, p0 = threadIdx.x >> 4;
  v4f s = {0.f, 0.f, 0.f, 0.f};
  if (col < hidden)
    for (int p = p0; p < nparts; p += 16)
      s += *reinterpret_cast<const v4f*>(parts + ((int64_t)p * 2 + which) * hidden + col);
  join[threadIdx.x] = s;
  __syncthreads();
  if (p0 != 0 || col >= hidden) return;
  for (int i = 1; i < 16; ++i) s += join[i * 16 + threadIdx.x];
  void* out = which ? dbias : dweight;
  if (f32) {
    v4f* o = reinterpret_cast<v4f*>((float*)out + col);
    *o = accumulate ? *o + s : s;
  } else {
    uint16_t* o = (uint16_t*)out + col;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = f32_to_bf16_rne(accumulate ? s[i] + bf16_to_f32(o[i]) : s[i]);
  }
}

bool bad_float(moe_float_fmt f) { return f != MOE_FLOAT_BF16 && f != MOE_FLOAT_F32; }
int64_t float_size(moe_float_fmt f) { return f == MOE_FLOAT_F32 ? 4 : 2; }
bool any_misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p % 16) return true;
  return false;
}

struct Buffer {
  const void* p;
  int64_t bytes;
};
// Does a written buffer share memory with another of the call's?
bool shared(std::initializer_list<Buffer> written, std::initializer_list<Buffer> read) {
  for (auto a = written.begin(); a != written.end(); ++a) {
    for (auto b = a + 1; b != written.end(); ++b)
      if (overlap(a->p, a->bytes, b->p, b->bytes)) return true;
    for (const Buffer& b : read)
      if (overlap(a->p, a->bytes, b.p, b.bytes)) return true;
  }
  return false;
}

moe_status check_sizes(int64_t rows, int hidden, int64_t x_stride, moe_float_fmt x_fmt,
                       moe_float_fmt w_fmt, moe_norm_kind kind,
                       const int32_t* psum_recv_per_rank, int num_src_ranks) {
  if (rows < 0 || rows > (1LL << 30) || hidden <= 0 || hidden % 8 != 0 || x_stride < hidden ||
      x_stride > (1LL << 30))
    return MOE_ERR_SHAPE;
  if (num_src_ranks < 0 || (psum_recv_per_rank && num_src_ranks == 0)) return MOE_ERR_SHAPE;
  if (bad_float(x_fmt) || bad_float(w_fmt) || (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) ||
      hidden > kMaxHidden)
    return MOE_ERR_UNSUPPORTED;
  if (x_stride * float_size(x_fmt) % 16) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Bytes of `rows` rows of x (the last one ends at its last column).
int64_t x_bytes(int64_t rows, int hidden, int64_t stride, moe_float_fmt f) {
  return rows > 0 ? ((rows - 1) * stride + hidden) * float_size(f) : 0;
}

template <bool kF32>
auto pick_norm(int hidden, int* per_block) {
  *per_block = hidden <= 2048 ? kWaves : 1;
  return hidden <= 512    ? norm_kernel<kF32, 1, 1>
         : hidden <= 1024 ? norm_kernel<kF32, 1, 2>
         : hidden <= 2048 ? norm_kernel<kF32, 1, 4>
         : hidden <= 4096 ? norm_kernel<kF32, kWaves, 2>
         : hidden <= 6144 ? norm_kernel<kF32, kWaves, 3>
                          : norm_kernel<kF32, kWaves, 4>;
}

template <bool kF32, bool kTwo, bool kSum>
auto pick_backward(int hidden) {
  return hidden <= 512    ? norm_backward_kernel<kF32, kTwo, kSum, 1, 1, 2>
         : hidden <= 2048 ? norm_backward_kernel<kF32, kTwo, kSum, 4, 1, 2>
         : hidden <= 4096 ? norm_backward_kernel<kF32, kTwo, kSum, 8, 1, 2>
                          : norm_backward_kernel<kF32, kTwo, kSum, 8, 2, 1>;
}
template <bool kF32>
auto pick_backward(int hidden, bool two, bool sum) {
  return two ? (sum ? pick_backward<kF32, true, true>(hidden)
                    : pick_backward<kF32, true, false>(hidden))
             : (sum ? pick_backward<kF32, false, true>(hidden)
                    : pick_backward<kF32, false, false>(hidden));
}

int64_t backward_grid(int64_t rows) { return rows < kParts ? rows : kParts; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_layer_norm(const void* x, int64_t x_stride, moe_float_fmt x_fmt,
                                     const void* branch, const void* weight, const void* bias,
                                     moe_float_fmt w_fmt, moe_norm_kind kind, float eps,
                                     const int32_t* psum_recv_per_rank, int num_src_ranks,
                                     int64_t rows, int hidden, void* sum, void* y, float* mean,
                                     float* rstd, void* stream) {
  const moe_status bad = check_sizes(rows, hidden, x_stride, x_fmt, w_fmt, kind,
                                     psum_recv_per_rank, num_src_ranks);
  if (bad != MOE_OK) return bad;
  if (!(eps >= 0.f) || __builtin_isinf(eps)) return MOE_ERR_SHAPE;
  if (!weight || (rows > 0 && (!x || !y))) return MOE_ERR_NULL;
  if (sum && !branch) return MOE_ERR_UNSUPPORTED;  // it would be x itself
  if (any_misaligned({x, branch, weight, bias, sum, y}) || (uintptr_t)mean % 4 ||
      (uintptr_t)rstd % 4)
    return MOE_ERR_ALIGNMENT;
  const int64_t n = rows * hidden, wide = n * float_size(x_fmt), gain = hidden * float_size(w_fmt);
  const bool in_place = sum == x && x_stride == hidden;
  const Buffer xb = {in_place ? nullptr : x, x_bytes(rows, hidden, x_stride, x_fmt)};
  if (shared({{sum, wide}, {y, n * 2}, {mean, rows * 4}, {rstd, rows * 4}},
             {xb,
              {branch, n * 2},
              {weight, gain},
              {bias, gain},
              {psum_recv_per_rank, num_src_ranks * 4LL}}) ||
      shared({{y, n * 2}, {mean, rows * 4}, {rstd, rows * 4}}, {{x, xb.bytes}}))
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  int per_block;
  auto kern = x_fmt == MOE_FLOAT_F32 ? pick_norm<true>(hidden, &per_block)
                                     : pick_norm<false>(hidden, &per_block);
  const int64_t blocks = (rows + per_block - 1) / per_block;
  const int64_t grid = blocks < 65536 ? blocks : 65536;  // grid-stride over the rest
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), x, x_stride, (const uint16_t*)branch,
                     weight, bias, w_fmt == MOE_FLOAT_F32, kind == MOE_NORM_RMS, eps,
                     psum_recv_per_rank, num_src_ranks, rows, hidden, sum, (uint16_t*)y, mean,
                     rstd);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

extern "C" size_t moe_layer_norm_backward_workspace_bytes(int64_t rows, int hidden) {
  if (rows < 0 || rows > (1LL << 30) || hidden <= 0 || hidden % 8 || hidden > kMaxHidden) return 0;
  return (size_t)backward_grid(rows) * 2 * hidden * sizeof(float);
}

extern "C" moe_status moe_layer_norm_backward(
    const void* dy, const void* dy2, const void* x, int64_t x_stride, moe_float_fmt x_fmt,
    const void* weight, moe_float_fmt w_fmt, moe_norm_kind kind, const float* mean,
    const float* rstd, const void* dsum, const int32_t* psum_recv_per_rank, int num_src_ranks,
    int64_t rows, int hidden, void* dx, void* dweight, void* dbias, moe_grad_fmt grad_fmt,
    int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status bad = check_sizes(rows, hidden, x_stride, x_fmt, w_fmt, kind,
                                     psum_recv_per_rank, num_src_ranks);
  if (bad != MOE_OK) return bad;
  if (grad_fmt != MOE_GRAD_BF16 && grad_fmt != MOE_GRAD_F32) return MOE_ERR_UNSUPPORTED;
  if (!weight || (rows > 0 && (!dy || !x || !rstd || !dx || (kind == MOE_NORM_LAYER && !mean))))
    return MOE_ERR_NULL;
  if (any_misaligned({dy, dy2, x, weight, dsum, dx, dweight, dbias}) || (uintptr_t)mean % 4 ||
      (uintptr_t)rstd % 4)
    return MOE_ERR_ALIGNMENT;
  const bool sums = dweight || dbias;
  const size_t need = sums ? moe_layer_norm_backward_workspace_bytes(rows, hidden) : 0;
  if (need && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  if (need && (uintptr_t)workspace % 256) return MOE_ERR_ALIGNMENT;
  const int64_t n = rows * hidden, wide = n * float_size(x_fmt), gain = hidden * float_size(w_fmt);
  const int64_t grad = hidden * (grad_fmt == MOE_GRAD_F32 ? 4 : 2);
  const Buffer ws = {need ? workspace : nullptr, (int64_t)need};
  if (shared({{dx, wide}, {dweight, grad}, {dbias, grad}, ws},
             {{dy, n * 2},
              {dy2, n * 2},
              {x, x_bytes(rows, hidden, x_stride, x_fmt)},
              {weight, gain},
              {mean, rows * 4},
              {rstd, rows * 4},
              {dx == dsum ? nullptr : dsum, wide},
              {psum_recv_per_rank, num_src_ranks * 4LL}}) ||
      shared({{dweight, grad}, {dbias, grad}, ws}, {{dsum, wide}}))
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0 && (accumulate || !sums)) return MOE_OK;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int64_t grid = backward_grid(rows);
  if (rows > 0) {
    auto kern = x_fmt == MOE_FLOAT_F32 ? pick_backward<true>(hidden, dy2, dsum)
                                       : pick_backward<false>(hidden, dy2, dsum);
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kBackThreads), 0, s, (const uint16_t*)dy,
                       (const uint16_t*)dy2, x, x_stride, weight, w_fmt == MOE_FLOAT_F32,
                       kind == MOE_NORM_RMS, mean, rstd, dsum, psum_recv_per_rank, num_src_ranks,
                       rows, hidden, wide > kCached, dx, sums ? (float*)workspace : nullptr);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH;
  }
  if (!sums) return MOE_OK;
  // dbias alone: the first sum is skipped by starting at the second.
  const dim3 g((hidden + 63) / 64, dbias && dweight ? 2 : 1);
  const float* parts = (const float*)workspace + (dweight ? 0 : hidden);
  hipLaunchKernelGGL(norm_join_kernel, g, dim3(256), 0, s, parts, (int)grid, hidden,
                     dweight ? dweight : dbias, dbias, grad_fmt == MOE_GRAD_F32,
                     accumulate != 0);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
