// The paged 8-bit cache: rotation of packed rows at any position, the append that rotates and
// quantises, and the way back to contiguous caches.  The attention over the pages is
// qd_paged_attn.cu.
#include <algorithm>
#include <atomic>

#include "qd_paged.cuh"

namespace qd {
namespace {

using paged::Cache;

// ------------------------------------------------------------------ angles
// The angle of a pair at a position is position * turns modulo 2^64, in units of 2^-64 turns: exact
// at any position, in one integer product.  Quadrant and remainder come off in integers too; sine
// and cosine of the remainder (at most pi/4) are the Taylor series in pairs of f32 (unevaluated
// sums h + l; off by 2^-43.9 and 2^-46.1 of themselves at most, over 24 million angles), so that after
// the last rounding they are the correctly rounded f32 values but for about one in 2^23.  That costs 300 f32 operations a pair of angles; FP64 units, of
// which this GPU has few, would take longer, and f32 alone is 2^-23 off, which moves a code of the
// cache in one of 10^5 and makes it depend on the side that computes it.
struct FF {
  float h, l;
};
__device__ __forceinline__ FF two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ FF quick_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ FF two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ FF mul(FF a, FF b) {
  FF p = two_prod(a.h, b.h);
  p.l = __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, p.l));
  return quick_sum(p.h, p.l);
}
// c + x, |c| >= |x.h|
__device__ __forceinline__ FF add(FF c, FF x) {
  const FF s = quick_sum(c.h, x.h);
  return quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(c.l, x.l)));
}

// (cos, sin) of pos * turns, times the magnitude, each rounded to f32.  Not inlined: its 300 instructions
// stand once in a kernel, which runs cold in a step of small calls.
__device__ __noinline__ float2 cos_sin(uint64_t turns, int pos, FF magnitude) {
  const uint64_t a = turns * (uint64_t)pos;
  const uint64_t quadrant = (a + (1ull << 61)) >> 62;
  const int64_t r = (int64_t)(a - (quadrant << 62));  // 2^-61 (pi / 4) each, at most 2^61 of them
  FF x;
  x.h = __ll2float_rn(r);
  x.l = __ll2float_rn(r - (int64_t)x.h);
  x.h *= 0x1p-61f;
  x.l *= 0x1p-61f;
  x = mul(x, {0x1.921fb6p-1f, -0x1.777a5cp-26f});  // pi / 4
  const FF z = mul(x, x);
  // sin x = x (1 + z (-1/3! + z (1/5! + z (-1/7! + z (1/9! - ...)))))
  float t = __fmaf_rn(z.h, -0x1.ae7f3ep-41f, 0x1.612462p-33f);
  t = __fmaf_rn(z.h, t, -0x1.ae6456p-26f);
  t = __fmaf_rn(z.h, t, 0x1.71de3ap-19f);
  FF s = quick_sum(-0x1.a01a02p-13f, __fmul_rn(z.h, t));
  s.l = __fadd_rn(s.l, 0x1.7f97fap-39f);
  s = add({0x1.111112p-7f, -0x1.dddddep-32f}, mul(z, s));
  s = add({-0x1.555556p-3f, 0x1.555556p-28f}, mul(z, s));
  s = add(x, mul(x, mul(z, s)));
  // cos x = 1 + z (-1/2! + z (1/4! + z (-1/6! + z (1/8! + ...))))
  t = __fmaf_rn(z.h, -0x1.93974ap-37f, 0x1.1eed8ep-29f);
  t = __fmaf_rn(z.h, t, -0x1.27e4fcp-22f);
  FF c = quick_sum(0x1.a01a02p-16f, __fmul_rn(z.h, t));
  c.l = __fadd_rn(c.l, -0x1.7f97fap-42f);
  c = add({-0x1.6c16c2p-10f, 0x1.27d27ep-35f}, mul(z, c));
  c = add({0x1.555556p-5f, -0x1.555556p-30f}, mul(z, c));
  c = add({-0.5f, 0.f}, mul(z, c));
  c = add({1.f, 0.f}, mul(z, c));
  s = mul(s, magnitude);
  c = mul(c, magnitude);
  const float cs = __fadd_rn(c.h, c.l), sn = __fadd_rn(s.h, s.l);
  switch ((int)quadrant & 3) {
    case 0: return make_float2(cs, sn);
    case 1: return make_float2(-sn, cs);
    case 2: return make_float2(-cs, -sn);
    default: return make_float2(sn, -cs);
  }
}

// a c - b s: where EXACT (both products in two parts; what the codes of keys are decided by) the rounded value but for
// the neighbour of about one in 2^24 (2 of 60 million, 20 of them with terms that cancel to 2^-25), else to 2^-24 of
// |b s| and of the result.  Queries and qd_rope_tokens are not EXACT: their values enter f32 arithmetic, and one product
// and a fused step take 8000 rows of 40 heads of 128 from 60 to 55 us (error against 64 bits 3.1e-8, rounded once 2.5e-8).
template <bool EXACT>
__device__ __forceinline__ float det(float a, float c, float b, float s) {
  if constexpr (!EXACT) return __fmaf_rn(a, c, -__fmul_rn(b, s));
  const FF p = two_prod(a, c), q = two_prod(b, s), d = two_sum(p.h, -q.h);
  const float r = __fadd_rn(d.h, __fadd_rn(d.l, __fsub_rn(p.l, q.l)));
  return isfinite(r) ? r : d.h;  // an infinity has no rest to add
}
__device__ __noinline__ float2 turn_small(float x0, float x1, float2 cs) {
  const double a = x0, b = x1;
  return make_float2((float)(a * cs.x - b * cs.y), (float)(a * cs.y + b * cs.x));
}
template <bool EXACT>
__device__ __forceinline__ void turn(float& x0, float& x1, float2 cs) {
  if constexpr (EXACT) {
    const float most = fmaxf(fabsf(x0), fabsf(x1));
    if (most < 0x1p-80f && most > 0.f) {  // the second parts would end at f32's smallest step
      const float2 y = turn_small(x0, x1, cs);
      x0 = y.x;
      x1 = y.y;
      return;
    }
  }
  const float y0 = det<EXACT>(x0, cs.x, x1, cs.y), y1 = det<EXACT>(x0, cs.y, -x1, cs.x);
  x0 = y0;
  x1 = y1;
}

// 8 elements of a head: the rotated ones are 4 pairs.  Unit u of a head has elements at [da, da + 4)
// and [db, db + 4); pairs 4u .. 4u + 3 where it is rotated.
struct Unit {
  int da, db;
  bool rotated;
};
__device__ __forceinline__ Unit unit_of(int u, int rot, int pairing) {
  Unit r;
  r.rotated = 8 * u < rot;
  const bool half = r.rotated && pairing == QD_ROPE_HALF;
  r.da = half ? 4 * u : 8 * u;
  r.db = half ? rot / 2 + 4 * u : 8 * u + 4;
  return r;
}
// cs: (cos, sin) of pairs 4u .. 4u + 3
template <bool EXACT>
__device__ __forceinline__ void turn_unit(float4& a, float4& b, const float2* cs, int pairing) {
  const float4 t0 = *reinterpret_cast<const float4*>(cs), t1 = *reinterpret_cast<const float4*>(cs + 2);
  const float2 c0 = make_float2(t0.x, t0.y), c1 = make_float2(t0.z, t0.w), c2 = make_float2(t1.x, t1.y),
               c3 = make_float2(t1.z, t1.w);
  if (pairing == QD_ROPE_HALF) {
    turn<EXACT>(a.x, b.x, c0);
    turn<EXACT>(a.y, b.y, c1);
    turn<EXACT>(a.z, b.z, c2);
    turn<EXACT>(a.w, b.w, c3);
  } else {
    turn<EXACT>(a.x, a.y, c0);
    turn<EXACT>(a.z, a.w, c1);
    turn<EXACT>(b.x, b.y, c2);
    turn<EXACT>(b.z, b.w, c3);
  }
}

struct Rotation {
  const uint64_t* turns;
  FF magnitude;
  int rot, pairing;
};
inline Rotation rotation_of(const uint64_t* turns, double magnitude, int rot, int pairing) {
  Rotation r;
  r.turns = turns;
  r.magnitude.h = (float)magnitude;
  r.magnitude.l = (float)(magnitude - (double)r.magnitude.h);
  r.rot = rot;
  r.pairing = pairing;
  return r;
}

// ------------------------------------------------------------------ rotation of packed rows
// y0 = x0 c - x1 s, y1 = x0 s + x1 c for the pairs of the first rot dimensions, the rest copied.
// A CTA takes a few rows: their angles once into shared memory, then a thread 8 elements at a time.
constexpr int kThreads = 256;
constexpr int kMaxRows = 16;                // of a CTA
constexpr int kMaxRot = 1024;
constexpr int kAngles = 2048;               // pairs of (cos, sin) of a CTA at most

struct RowsArgs {
  const float* x;
  int64_t x_stride;
  float* out;
  int64_t out_stride;
  int n_tokens, n_heads, hd, rows;  // rows: of a CTA
  uint32_t heads_magic;             // 2^32 / n_heads rounded up; not looked at with one row or head
  Rotation rot;
};

// Rows first .. of this CTA; find() puts the position of each into s_pos, < 0: not written.  A thread keeps
// its unit of a head and goes from one (row, head) to another, four at a time, whose loads are on their way
// while the CTA finds the positions and makes the angles.
template <typename Find>
__device__ __forceinline__ void rotate_rows(const RowsArgs& a, int first, int* s_pos, float2* s_cs, Find find) {
  const int n = min(a.rows, a.n_tokens - first), pairs = a.rot.rot / 2, per = a.hd / 8;
  const int groups = kThreads / per, group = threadIdx.x / per, at = threadIdx.x - group * per;
  const int items = group < groups ? n * a.n_heads : 0;  // the last threads have no whole group
  const Unit u = unit_of(at, a.rot.rot, a.rot.pairing);
  const bool copies = u.rotated || a.x != a.out;  // in place, what is not rotated stays
  constexpr int kAtOnce = 4;
  bool angles = false;
  for (int j0 = group; j0 < items || !angles; j0 += kAtOnce * groups) {
    float4 v0[kAtOnce], v1[kAtOnce];
    int row[kAtOnce], head[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int j = j0 + i * groups;
      row[i] = -1;
      if (j >= items || !copies) continue;
      const int r = a.rows == 1 ? 0 : a.n_heads == 1 ? j : (int)__umulhi((uint32_t)j, a.heads_magic);
      head[i] = j - r * a.n_heads;
      row[i] = r;
      const float* src = a.x + (int64_t)(first + r) * a.x_stride + head[i] * a.hd;
      v0[i] = __ldcg(reinterpret_cast<const float4*>(src + u.da));
      v1[i] = __ldcg(reinterpret_cast<const float4*>(src + u.db));
    }
    if (!angles) {  // every thread comes here once
      find(n);
      __syncthreads();
      for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
        const int r = i / pairs, p = s_pos[r];
        if (p >= 0) s_cs[i] = cos_sin(__ldg(a.rot.turns + (i - r * pairs)), p, a.rot.magnitude);
      }
      __syncthreads();
      angles = true;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (row[i] < 0 || s_pos[row[i]] < 0) continue;
      if (u.rotated) turn_unit<false>(v0[i], v1[i], s_cs + row[i] * pairs + 4 * at, a.rot.pairing);
      float* dst = a.out + (int64_t)(first + row[i]) * a.out_stride + head[i] * a.hd;
      *reinterpret_cast<float4*>(dst + u.da) = v0[i];
      *reinterpret_cast<float4*>(dst + u.db) = v1[i];
    }
  }
}
inline uint32_t magic_of(int n) { return n < 2 ? 0u : (uint32_t)(((1ull << 32) + n - 1) / n); }

__global__ void __launch_bounds__(kThreads) k_rope_tokens(RowsArgs a, const int32_t* __restrict__ pos) {
  __shared__ __align__(16) float2 s_cs[kAngles];
  __shared__ int s_pos[kMaxRows];
  const int first = blockIdx.x * a.rows;
  rotate_rows(a, first, s_pos, s_cs, [&](int n) {
    if (threadIdx.x < n) s_pos[threadIdx.x] = pos[first + threadIdx.x];
  });
}

// Rows of a CTA: about 2560 units (10 a thread; 8000 rows of 40 heads of 128 53.2 us with half, 51.2 so, 56.2 with twice as many), one row while there are SMs without one.
inline int rows_per_cta(int n_tokens, int n_heads, int hd, int rot) {
  const int units = n_heads * (hd / 8);
  int rows = std::min({kMaxRows, kAngles / (rot / 2), std::max(2560 / units, 1)});
  while (rows > 1 && (n_tokens + rows - 1) / rows < 4 * attn_sm_count()) rows /= 2;
  return rows;
}

// ------------------------------------------------------------------ append
// Per block of 16 positions and head: s = max(s before, max |x| / top), code = nearest(x / s), and
// where s grows the codes before are rounded again.  A CTA takes a block of one sequence and some
// heads: the angles of its rows once into shared memory, then a warp a (head, K or V) at a time,
// whole in registers between its maximum and its codes.  More CTAs rotate the queries.
struct AppendArgs {
  Cache c;
  const float *q, *k, *v;
  int64_t stride;
  const int32_t *row_start, *pos;
  int n_seqs, n_tokens;
  int splits, heads;  // CTAs of a block, heads of each
  int kv_ctas;
  RowsArgs rows;      // of q
};

template <int FMT>
__device__ __forceinline__ constexpr float top_code() {
  return FMT == QD_KV_I8 ? 127.f : 448.f;
}
// Codes of four values, given value / scale.
template <int FMT>
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {
  if constexpr (FMT == QD_KV_I8) {
    auto one = [](float x) { return (uint32_t)(int)fminf(fmaxf(roundf(x), -127.f), 127.f) & 0xFFu; };
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
  } else {
    uint16_t lo, hi;  // the first operand becomes the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
  }
}
template <int FMT>
__device__ __forceinline__ float4 values_of(uint32_t w) {
  if constexpr (FMT == QD_KV_I8) {
    return make_float4((float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24));
  } else {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(x.x, x.y, y.x, y.y);
  }
}
// The same of eight values, given 1 / scale to the nearest: x (1 / scale) is within 1.5 * 2^-23 of the
// rounded quotient, relatively.  False where that could matter, and the quotients have to be formed.
template <int FMT>
__device__ __forceinline__ bool codes_by(float4 x, float4 y, float inv, uint32_t& w0, uint32_t& w1) {
  if constexpr (FMT == QD_KV_I8) {
    constexpr float kMagic15 = 12582912.f;  // 1.5 * 2^23: a sum's low byte is the nearest whole number
    float far = 0.f;
    auto one = [&](float v) {
      const float t = v * inv, m = __fadd_rn(t, kMagic15);
      far = fmaxf(far, fabsf(t - __fsub_rn(m, kMagic15)));
      return __float_as_uint(m);
    };
    auto four = [&](float4 v) {
      return __byte_perm(__byte_perm(one(v.x), one(v.y), 0x0040u), __byte_perm(one(v.z), one(v.w), 0x0040u), 0x5410u);
    };
    w0 = four(x);
    w1 = four(y);
    return far < 0.49996f;  // 127 * 1.5 * 2^-23 < 2.3e-5 from a tie
  } else {
    const float up = inv * (1.f + 0x1p-21f), down = inv * (1.f - 0x1p-21f);
    w0 = codes_of<FMT>(x.x * up, x.y * up, x.z * up, x.w * up);
    w1 = codes_of<FMT>(y.x * up, y.y * up, y.z * up, y.w * up);
    return w0 == codes_of<FMT>(x.x * down, x.y * down, x.z * down, x.w * down) &&
           w1 == codes_of<FMT>(y.x * down, y.y * down, y.z * down, y.w * down);
  }
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t abs_max(float4 x) {
  return max(max(abs_bits(x.x), abs_bits(x.y)), max(abs_bits(x.z), abs_bits(x.w)));
}

// Blocks that sequence b appends to, and its first position.
__device__ __forceinline__ int blocks_of(const AppendArgs& a, int b, int& p0) {
  int first;
  const int t = paged::rows_of(a.row_start, b, a.n_tokens, first);
  p0 = a.pos[b];
  if (t == 0 || p0 < 0 || p0 >= a.c.capacity) return 0;
  return (min((int64_t)p0 + t, (int64_t)a.c.capacity) - 1) / QD_KV_BLOCK - p0 / QD_KV_BLOCK + 1;
}

// With more than this many CTAs of them to an SM, the queries have a launch of their own, whose CTAs need
// fewer registers.
constexpr int kQueriesApart = 2;
// Rows first .. of the queries, rotated by their sequences' positions.
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int first, int* s_pos, float2* s_cs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  rotate_rows(a.rows, first, s_pos, s_cs, [&](int n) {
    for (int r = warp; r < n; r += kThreads / 32) {  // the last sequence that starts at or before the row
      const int row = first + r;
      int before = 0;
      for (int b = lane; b < a.n_seqs; b += 32) before += a.row_start[b] <= row;
      before = __reduce_add_sync(0xffffffffu, before);
      if (lane == 0) {
        int p = -1;
        if (before && row < a.row_start[before]) {
          const int p0 = a.pos[before - 1];
          if (p0 >= 0 && p0 <= a.c.capacity) p = p0 + (row - a.row_start[before - 1]);
        }
        s_pos[r] = p;
      }
    }
  });
}
__global__ void __launch_bounds__(kThreads) k_paged_queries(AppendArgs a) {
  __shared__ __align__(16) float2 s_cs[kAngles];
  __shared__ int s_pos[kMaxRows];
  rotate_queries(a, blockIdx.x * a.rows.rows, s_pos, s_cs);
}

// f32 values of a warp's block on their way: rows of HD + 4, so that neighbouring slots meet other banks.
template <int HD>
constexpr int kBlockFloats = 16 * (HD + 4);

template <int HD, int FMT>
__global__ void __launch_bounds__(kThreads, 3) k_paged_append(AppendArgs a) {
  extern __shared__ __align__(16) float s_values[];
  __shared__ __align__(16) float2 s_cs[kAngles];
  __shared__ int s_pos[kMaxRows];
  __shared__ int s_seq, s_block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= a.kv_ctas) {
    rotate_queries(a, (blockIdx.x - a.kv_ctas) * a.rows.rows, s_pos, s_cs);
    return;
  }
  const int unit = blockIdx.x / a.splits, h0 = blockIdx.x % a.splits * a.heads;
  if (warp == 0) {  // the sequence of the unit: blocks counted up, 32 sequences at a time
    int base = 0, seq = -1, block = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
      int p0 = 0;
      const int n = b0 + lane < a.n_seqs ? blocks_of(a, b0 + lane, p0) : 0;
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const unsigned over = __ballot_sync(0xffffffffu, base + sum > unit);
      if (over) {
        const int l = __ffs(over) - 1;
        seq = b0 + l;
        block = __shfl_sync(0xffffffffu, p0 / QD_KV_BLOCK + unit - (base + sum - n), l);
        break;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      s_seq = seq;
      s_block = block;
    }
  }
  __syncthreads();
  const int seq = s_seq, block = s_block;
  if (seq < 0) return;
  int row0;
  const int t = paged::rows_of(a.row_start, seq, a.n_tokens, row0);
  const int p0 = a.pos[seq];
  const int lo = max(block * QD_KV_BLOCK, p0) - block * QD_KV_BLOCK;  // slots of new rows
  const int hi = (int)min((int64_t)p0 + t - (int64_t)block * QD_KV_BLOCK, (int64_t)QD_KV_BLOCK);
  const int64_t src0 = row0 + ((int64_t)block * QD_KV_BLOCK - p0);  // row of slot 0
  const int heads = min(a.heads, a.c.n_kv - h0);
  float* mine = s_values + warp * kBlockFloats<HD>;
  auto fetch = [&](int task) {  // the new rows of (head, K or V) into this warp's block
    const float* src = (task & 1 ? a.v : a.k) + (int64_t)(h0 + (task >> 1)) * HD;
#pragma unroll 4
    for (int i = lane; i < 16 * HD / 4; i += 32) {
      const int slot = i / (HD / 4), c = i % (HD / 4);
      if (slot >= lo && slot < hi) {
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(mine + slot * (HD + 4) + 4 * c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + (src0 + slot) * a.stride + 4 * c)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (warp < 2 * heads) fetch(warp);  // under the angles
  int in_page;
  const int page = paged::page_of(a.c, paged::table_row(a.c, seq), block, in_page);
  if (page < 0) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    return;
  }
  const int pairs = a.rows.rot.rot / 2;
  for (int i = threadIdx.x; i < (hi - lo) * pairs; i += kThreads) {
    const int r = i / pairs, j = i - r * pairs;
    s_cs[(lo + r) * (pairs + 2) + j] = cos_sin(__ldg(a.rows.rot.turns + j), block * QD_KV_BLOCK + lo + r, a.rows.rot.magnitude);
  }
  __syncthreads();

  // A lane has units 2 i + (lane & 1) of slot lane / 2, so that a warp's lanes rotate together or not at
  // all.  The loops are not unrolled: a block's rotation unrolled is 30 KB of code, whose fetching took
  // longer than its running (40 us for 6000 rows of 8 heads of 128, and 28 so).
  const int slot = lane >> 1;
  const bool live = slot >= lo && slot < hi;
  for (int task = warp; task < 2 * heads; task += kThreads / 32) {
    const bool isv = task & 1;
    const int rot = isv ? 0 : a.rows.rot.rot;
    const int64_t at = paged::block_index(a.c, page, h0 + (task >> 1), in_page);
    float* scale = (isv ? a.c.vs : a.c.ks) + at;
    uint8_t* codes = (isv ? a.c.v : a.c.k) + at * (16 * HD);
    if (task != warp) fetch(task);
    const float old = lo > 0 ? *scale : 0.f;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    float* row = mine + slot * (HD + 4);
    uint32_t most = 0;
    if (live) {
#pragma unroll 1
      for (int u = lane & 1; u < HD / 8; u += 2) {
        const Unit w = unit_of(u, rot, a.rows.rot.pairing);
        float4 x = *reinterpret_cast<const float4*>(row + w.da), y = *reinterpret_cast<const float4*>(row + w.db);
        if (w.rotated) {
          turn_unit<true>(x, y, s_cs + slot * (pairs + 2) + 4 * u, a.rows.rot.pairing);
          *reinterpret_cast<float4*>(row + w.da) = x;
          *reinterpret_cast<float4*>(row + w.db) = y;
        }
        most = max(most, max(abs_max(x), abs_max(y)));
      }
    }
    __syncwarp();  // half of what a lane reads below its neighbour has rotated; the reduction orders no memory
    most = __reduce_max_sync(0xffffffffu, most);
    const bool broken = most >= 0x7F800000u || isnan(old);
    const float top = __fdiv_rn(__uint_as_float(most), top_code<FMT>());
    const float now = broken ? __uint_as_float(0x7FC00000u) : fmaxf(old, top), inv = __frcp_rn(now);
    if (live) {
#pragma unroll 1
      for (int u = lane & 1; u < HD / 8; u += 2) {
        const float4 x = *reinterpret_cast<const float4*>(row + 8 * u), y = *reinterpret_cast<const float4*>(row + 8 * u + 4);
        uint32_t w0 = 0, w1 = 0;
        if (now > 0.f && !(now >= 0x1p-100f && codes_by<FMT>(x, y, inv, w0, w1))) {
          w0 = codes_of<FMT>(__fdiv_rn(x.x, now), __fdiv_rn(x.y, now), __fdiv_rn(x.z, now), __fdiv_rn(x.w, now));
          w1 = codes_of<FMT>(__fdiv_rn(y.x, now), __fdiv_rn(y.y, now), __fdiv_rn(y.z, now), __fdiv_rn(y.w, now));
        }
        *reinterpret_cast<uint2*>(codes + slot * HD + 8 * u) = make_uint2(w0, w1);
      }
    }
    __syncwarp();  // the block has been read
    if (lo > 0 && now > old) {  // the codes before, in the new steps
      for (int i = lane; i < lo * HD / 4; i += 32) {
        uint32_t* w = reinterpret_cast<uint32_t*>(codes) + i;
        const float4 c = values_of<FMT>(*w);
        auto again = [&](float v) { return __fdiv_rn(__fmul_rn(v, old), now); };
        *w = codes_of<FMT>(again(c.x), again(c.y), again(c.z), again(c.w));
      }
    }
    if (lane == 0) *scale = now;
  }
}

// ------------------------------------------------------------------ read back
// value = code * scale, once rounded to f32 and for binary16 once more.  A warp takes a block of 16
// positions of one head, 16 codes a lane and step.
__device__ __forceinline__ void put16(float* p, const float4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = v[i];
}
__device__ __forceinline__ void put16(__half* p, const float4 (&v)[4]) {
  __half2 h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = __floats2half2_rn(v[i].x, v[i].y);
    h[2 * i + 1] = __floats2half2_rn(v[i].z, v[i].w);
  }
  reinterpret_cast<uint4*>(p)[0] = reinterpret_cast<const uint4*>(h)[0];
  reinterpret_cast<uint4*>(p)[1] = reinterpret_cast<const uint4*>(h)[1];
}

template <int HD, int FMT, typename OUT>
__global__ void __launch_bounds__(kThreads) k_paged_read(Cache c, const int32_t* __restrict__ len, int max_ctx,
                                                         int blocks, OUT* __restrict__ k_out, OUT* __restrict__ v_out) {
  const int seq = blockIdx.z, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // (block, head), heads fastest
  const int n = min(len[seq], min(max_ctx, c.capacity));
  const int block = unit / c.n_kv, head = unit - block * c.n_kv;
  if (block >= blocks || block * QD_KV_BLOCK >= n) return;
  int in_page;
  const int page = paged::page_of(c, paged::table_row(c, seq), block, in_page);
  const int64_t at = page < 0 ? 0 : paged::block_index(c, page, head, in_page);
  const bool isv = blockIdx.y;
  const float scale = page < 0 ? __uint_as_float(0x7FC00000u) : (isv ? c.vs : c.ks)[at];
  const uint4* src = reinterpret_cast<const uint4*>((isv ? c.v : c.k) + at * (16 * HD));
  OUT* dst = (isv ? v_out : k_out) + (((int64_t)seq * c.n_kv + head) * max_ctx + block * QD_KV_BLOCK) * HD;
  const int live = min(n - block * QD_KV_BLOCK, QD_KV_BLOCK) * HD;
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) {
    const int e = 16 * (lane + 32 * i);
    if (e >= live) break;
    const uint4 w = src[lane + 32 * i];
    float4 v[4] = {values_of<FMT>(w.x), values_of<FMT>(w.y), values_of<FMT>(w.z), values_of<FMT>(w.w)};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float4(v[j].x * scale, v[j].y * scale, v[j].z * scale, v[j].w * scale);
    put16(dst + e, v);
  }
}

inline qd_status rotation_status(int head_dim, int rot_dim, const uint64_t* turns, double magnitude,
                                 qd_rope_pairing pairing) {
  if (!turns || !std::isfinite(magnitude) || !std::isfinite((float)magnitude)) return QD_ERR_INVALID_ARG;
  if (pairing != QD_ROPE_ADJACENT && pairing != QD_ROPE_HALF) return QD_ERR_UNSUPPORTED;
  if (rot_dim < 8 || rot_dim % 8 || rot_dim > head_dim) return QD_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(turns) & 7) return QD_ERR_ALIGN;
  return QD_OK;
}

template <int HD, int FMT>
qd_status launch_append(const AppendArgs& a, int ctas, cudaStream_t st) {
  constexpr int kSmem = kThreads / 32 * kBlockFloats<HD> * 4;
  static std::atomic<bool> done[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QD_ERR_CUDA;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(k_paged_append<HD, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return QD_ERR_CUDA;
    done[dev] = true;
  }
  k_paged_append<HD, FMT><<<ctas, kThreads, kSmem, st>>>(a);
  return launch_status();
}

template <int HD, int FMT>
qd_status launch_read(const Cache& c, const int32_t* len, int n_seqs, int max_ctx, void* k_out, void* v_out, int f16,
                      cudaStream_t st) {
  const int blocks = (std::min(max_ctx, c.capacity) + QD_KV_BLOCK - 1) / QD_KV_BLOCK;
  const int64_t units = (int64_t)blocks * c.n_kv;
  const dim3 grid((unsigned)((units + kThreads / 32 - 1) / (kThreads / 32)), 2, (unsigned)n_seqs);
  if (f16)
    k_paged_read<HD, FMT><<<grid, kThreads, 0, st>>>(c, len, max_ctx, blocks, static_cast<__half*>(k_out),
                                                     static_cast<__half*>(v_out));
  else
    k_paged_read<HD, FMT><<<grid, kThreads, 0, st>>>(c, len, max_ctx, blocks, static_cast<float*>(k_out),
                                                     static_cast<float*>(v_out));
  return launch_status();
}

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_rope_plan(double theta, int rot_dim, qd_rope_scaling scaling, double factor, int trained_ctx, double low,
                       double high, uint64_t* turns_host, double* magnitude_host) {
  if (!turns_host || !magnitude_host) return QD_ERR_INVALID_ARG;
  if (scaling < QD_ROPE_SCALE_NONE || scaling > QD_ROPE_SCALE_PAIRS) return QD_ERR_UNSUPPORTED;
  if (rot_dim < 8 || rot_dim % 8 || rot_dim > kMaxRot) return QD_ERR_SHAPE;
  if (!std::isfinite(theta) || theta <= 1.0) return QD_ERR_INVALID_ARG;
  const bool blend = scaling == QD_ROPE_SCALE_TURNS || scaling == QD_ROPE_SCALE_PAIRS;
  if (scaling != QD_ROPE_SCALE_NONE && (!std::isfinite(factor) || factor < 1.0)) return QD_ERR_INVALID_ARG;
  if (blend && (trained_ctx < 1 || !std::isfinite(high) || !(low > 0.0) || !(high > low))) return QD_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  double first = 0, last = 0;
  if (scaling == QD_ROPE_SCALE_NTK) theta *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  if (!std::isfinite(theta)) return QD_ERR_INVALID_ARG;
  if (scaling == QD_ROPE_SCALE_PAIRS) {
    auto at = [&](double turns) { return rot_dim * std::log(trained_ctx / (two_pi * turns)) / (2 * std::log(theta)); };
    first = std::max(std::floor(at(high)), 0.0);
    last = std::min(std::ceil(at(low)), rot_dim - 1.0);
  }
  *magnitude_host = scaling == QD_ROPE_SCALE_PAIRS ? 0.1 * std::log(factor) + 1.0 : 1.0;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == QD_ROPE_SCALE_LINEAR) f /= factor;
    if (blend) {
      double w = scaling == QD_ROPE_SCALE_TURNS ? (trained_ctx * f / two_pi - low) / (high - low)
                                                : 1.0 - (i - first) / std::max(last - first, 0.001);
      w = std::min(std::max(w, 0.0), 1.0);
      f = f * (w + (1.0 - w) / factor);
    }
    // f / (2 pi), the reciprocal in two doubles, to the nearest 2^-64
    const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    const double p = f * hi, rest = std::fma(f, hi, -p) + f * lo;
    const double whole = std::floor(std::ldexp(p, 64));
    turns_host[i] = (uint64_t)whole + (uint64_t)(int64_t)std::llrint((std::ldexp(p, 64) - whole) + std::ldexp(rest, 64));
  }
  return QD_OK;
}

qd_status qd_rope_tokens(const float* x, int64_t x_stride, float* out, int64_t out_stride, int n_tokens, int n_heads,
                         int head_dim, int rot_dim, const int32_t* pos, qd_rope_pairing pairing, const uint64_t* turns,
                         double magnitude, qd_stream_t stream) {
  if (!x || !out || !pos) return QD_ERR_INVALID_ARG;
  if (n_tokens < 1 || n_tokens > QD_MAX_GEMM_TOKENS || n_heads < 1 || n_heads > 65536 || head_dim < 8 ||
      head_dim % 8 || head_dim > 1024)
    return QD_ERR_SHAPE;
  const qd_status r = rotation_status(head_dim, rot_dim, turns, magnitude, pairing);
  if (r != QD_OK) return r;
  const int64_t row = (int64_t)n_heads * head_dim;
  if (n_tokens > 1 && (x_stride < row || out_stride < row)) return QD_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(out) || !aligned4(pos)) return QD_ERR_ALIGN;
  if (n_tokens > 1 && (x_stride % 4 || out_stride % 4)) return QD_ERR_ALIGN;
  if (x == out && n_tokens > 1 && x_stride != out_stride) return QD_ERR_INVALID_ARG;
  const RowsArgs a = {x, x_stride, out, out_stride, n_tokens, n_heads, head_dim,
                      rows_per_cta(n_tokens, n_heads, head_dim, rot_dim), magic_of(n_heads),
                      rotation_of(turns, magnitude, rot_dim, pairing)};
  k_rope_tokens<<<(n_tokens + a.rows - 1) / a.rows, kThreads, 0, (cudaStream_t)stream>>>(a, pos);
  return launch_status();
}

qd_status qd_paged_append(const qd_paged_kv* kv, const float* q, const float* k, const float* v, int64_t token_stride,
                          float* q_out, int n_heads, int n_tokens, const int32_t* row_start, const int32_t* pos,
                          int n_seqs, int rot_dim, qd_rope_pairing pairing, const uint64_t* turns, double magnitude,
                          qd_stream_t stream) {
  if (!k || !v || !row_start || !pos || (q && !q_out)) return QD_ERR_INVALID_ARG;
  qd_status r = paged::cache_status(kv, n_seqs);
  if (r != QD_OK) return r;
  if (n_tokens < 1 || n_tokens > QD_MAX_GEMM_TOKENS || (q && (n_heads < 1 || n_heads > 65536))) return QD_ERR_SHAPE;
  r = rotation_status(kv->head_dim, rot_dim, turns, magnitude, pairing);
  if (r != QD_OK) return r;
  const int64_t widest = (int64_t)std::max(q ? n_heads : 0, kv->n_kv_heads) * kv->head_dim;
  if (n_tokens > 1 && token_stride < widest) return QD_ERR_SHAPE;
  if ((q && (!aligned16(q) || !aligned16(q_out))) || !aligned16(k) || !aligned16(v) || !aligned4(row_start) ||
      !aligned4(pos))
    return QD_ERR_ALIGN;
  if (n_tokens > 1 && token_stride % 4) return QD_ERR_ALIGN;
  AppendArgs a;
  a.c = paged::cache_of(kv);
  a.q = q;
  a.k = k;
  a.v = v;
  a.stride = token_stride;
  a.row_start = row_start;
  a.pos = pos;
  a.n_seqs = n_seqs;
  a.n_tokens = n_tokens;
  // t rows touch at most min(t, (t + 30) / 16) blocks
  const int units = (int)std::min<int64_t>(n_tokens, (n_tokens + 30ll * n_seqs) / QD_KV_BLOCK);
  a.splits = std::max(1, std::min((kv->n_kv_heads + 3) / 4, (4 * attn_sm_count() + units - 1) / units));
  a.heads = (kv->n_kv_heads + a.splits - 1) / a.splits;
  a.splits = (kv->n_kv_heads + a.heads - 1) / a.heads;
  a.kv_ctas = units * a.splits;
  const int qh = q ? n_heads : 1;
  a.rows = {q, token_stride, q_out, (int64_t)qh * kv->head_dim, n_tokens, qh, kv->head_dim,
            rows_per_cta(n_tokens, qh, kv->head_dim, rot_dim), magic_of(qh),
            rotation_of(turns, magnitude, rot_dim, pairing)};
  cudaStream_t st = (cudaStream_t)stream;
  const int q_ctas = q ? (n_tokens + a.rows.rows - 1) / a.rows.rows : 0;
  const bool apart = q_ctas > kQueriesApart * attn_sm_count();
  if (apart) {
    k_paged_queries<<<q_ctas, kThreads, 0, st>>>(a);
    r = launch_status();
    if (r != QD_OK) return r;
  }
  const int ctas = a.kv_ctas + (apart ? 0 : q_ctas);
  if (kv->head_dim == 64)
    return kv->fmt == QD_KV_I8 ? launch_append<64, QD_KV_I8>(a, ctas, st) : launch_append<64, QD_KV_E4M3>(a, ctas, st);
  return kv->fmt == QD_KV_I8 ? launch_append<128, QD_KV_I8>(a, ctas, st) : launch_append<128, QD_KV_E4M3>(a, ctas, st);
}

qd_status qd_paged_read(const qd_paged_kv* kv, const int32_t* len, int n_seqs, int max_ctx, void* k_out, void* v_out,
                        int out_f16, qd_stream_t stream) {
  if (!len || !k_out || !v_out || (out_f16 != 0 && out_f16 != 1)) return QD_ERR_INVALID_ARG;
  const qd_status r = paged::cache_status(kv, n_seqs);
  if (r != QD_OK) return r;
  if (max_ctx < 1 || max_ctx > (1 << 30)) return QD_ERR_SHAPE;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(len)) return QD_ERR_ALIGN;
  const Cache c = paged::cache_of(kv);
  if ((int64_t)((std::min(max_ctx, c.capacity) + 15) / 16) * c.n_kv > (1ll << 31) - 1) return QD_ERR_SHAPE;
  cudaStream_t st = (cudaStream_t)stream;
  if (kv->head_dim == 64)
    return kv->fmt == QD_KV_I8 ? launch_read<64, QD_KV_I8>(c, len, n_seqs, max_ctx, k_out, v_out, out_f16, st)
                               : launch_read<64, QD_KV_E4M3>(c, len, n_seqs, max_ctx, k_out, v_out, out_f16, st);
  return kv->fmt == QD_KV_I8 ? launch_read<128, QD_KV_I8>(c, len, n_seqs, max_ctx, k_out, v_out, out_f16, st)
                             : launch_read<128, QD_KV_E4M3>(c, len, n_seqs, max_ctx, k_out, v_out, out_f16, st);
}

}  // extern "C"
