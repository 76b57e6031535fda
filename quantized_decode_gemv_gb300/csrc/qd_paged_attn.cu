// Causal attention of packed rows over the pages of an 8-bit cache:
//   o = sum_j softmax_j(scale q . k_j) v_j,  k_j = code * scale of its block, over the positions
// j = 0 .. p of a row at position p (the last `window` of them with a window).
//
// The rows that share a kv head (tokens x query heads of the group) walk its positions together
// with an online softmax: s = q k^T and o += p v are matrix products with f32 accumulators.  Codes
// of 8 bits are exact in binary16, so they enter the products as they are; a block's scale of keys
// multiplies its scores, that of values its weights.  Outputs are f32 and meant to be as exact as f32
// arithmetic, so queries and weights enter in two binary16 parts, hi = rn(x), lo = rn(x - hi), at a power of
// two that puts the largest of a row of queries at 2^14 to 2^15 and the largest weight times scale at
// 2^12 to 2^15: what is 2^-15 of that or more keeps 22 bits, what is less is 2^-38 of it off.  The matrix units
// cut their f32 sums off instead of rounding them: a tile's products start from zero and are added
// to o with rounded f32 additions.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "qd_paged.cuh"
#include "qd_tc.cuh"

namespace qd {
namespace {

using paged::Cache;

constexpr float kBias = 14.f;  // log2 of the weights' scale
constexpr int kStart = 1;      // what the start of a walk costs, in units
constexpr int kMinPer = 2;     // units of a CTA at least
constexpr int kWholeUnits = 4; // walks of at most so many units are not cut

struct AttnArgs {
  Cache c;
  const float* q;
  int64_t q_stride;
  float* out;
  int n_heads, n_tokens, n_seqs, group;
  const int32_t *row_start, *pos;
  float scale;  // times log2 e: scores in log2 units
  int window;
  int whole;     // units to a walk where no walk is cut, 0: the walks are cut evenly
  int max_rows;  // sequences of more rows (tokens x group) are another kernel's
  float* ws;
};

// ------------------------------------------------------------------ building blocks
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {  // 16 zero bytes if not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
template <int TO, int FROM>
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(TO), "n"(FROM) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.u32 p, %2, 0;\n"
      "@p cp.async.ca.shared.global [%0], [%1], 4;\n"
      "}\n" ::"r"(dst),
      "l"(src), "r"((uint32_t)live)
      : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// (x, y) -> two binary16 parts, hi = rn(x), lo = rn(x - hi)
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t abs_max(float4 x) {
  return max(max(abs_bits(x.x), abs_bits(x.y)), max(abs_bits(x.z), abs_bits(x.w)));
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 .. 127
// Exponent e of a largest magnitude (given by its bits), so that x 2^-e is in 2^14 .. 2^15 (less for
// one under 2^-100); an infinity or NaN stays what it is.
__device__ __forceinline__ int scale_exp(uint32_t abs_bits) {
  return min(max((int)(abs_bits >> 23) - 127, -100), 127) - 14;
}

// Four codes -> two binary16 pairs (codes 0, 1 and 2, 3), exactly.
template <int FMT>
__device__ __forceinline__ void to_h2x2(uint32_t w, uint32_t& h01, uint32_t& h23) {
  if constexpr (FMT == QD_KV_I8) {
    tc::i8x4_to_h2x2(w, h01, h23);
  } else {
    asm("{\n"
        ".reg .b16 lo, hi;\n"
        "mov.b32 {lo, hi}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n"
        "}\n"
        : "=r"(h01), "=r"(h23)
        : "r"(w));
  }
}

// ------------------------------------------------------------------ plan
// The walks of all (sequence, kv head, block of BM rows) are laid end to end in units of W tiles
// and cut evenly over the CTAs, whatever the lengths; a walk's start counts as kStart units.
template <int W>
struct Plan {
  int64_t off[QD_MAX_SEQS + 1];  // first unit of each sequence
  int64_t sums[W];
};
// A sequence's tokens, the first one's row and position: -2 where the positions are out of range (zeros).
__device__ __forceinline__ int tokens_of(const AttnArgs& a, int b, int& row0, int& p0) {
  const int t = paged::rows_of(a.row_start, b, a.n_tokens, row0);
  p0 = a.pos[b];
  if (p0 < 0 || (int64_t)p0 + t > a.c.capacity) p0 = -2;
  return t;
}

struct Walk {  // of one sequence
  int first_tile, nt, rb, len;
};
template <int TILE, int W, int BM>
__device__ __forceinline__ Walk walk_of(const AttnArgs& a, int p0, int t) {
  Walk w = {0, 0, 0, 0};
  const int64_t rows = (int64_t)t * a.group;
  if (t == 0 || rows > a.max_rows) return w;
  w.rb = (int)((rows + BM - 1) / BM);
  w.nt = 1;
  if (p0 >= 0) {
    w.first_tile = a.window > 0 ? max(p0 - a.window + 1, 0) / TILE : 0;
    w.nt = ((p0 + t - 1) / TILE - w.first_tile) / W + 1;
  }
  w.len = a.whole ? a.whole : w.nt + kStart;
  return w;
}

// Filled by the whole CTA of W warps.
template <int TILE, int W, int BM>
__device__ __forceinline__ void make_plan(const AttnArgs& a, Plan<W>* p) {
  constexpr int kPer = QD_MAX_SEQS / (32 * W);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t mine[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = threadIdx.x * kPer + i;
    mine[i] = 0;
    if (b < a.n_seqs) {
      int row0, p0;
      const int t = tokens_of(a, b, row0, p0);
      const Walk w = walk_of<TILE, W, BM>(a, p0, t);
      mine[i] = (int64_t)w.len * w.rb * a.c.n_kv;
    }
    sum += mine[i];
  }
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) p->sums[warp] = upto;
  __syncthreads();
  int64_t at = upto - sum;
#pragma unroll
  for (int w = 0; w < W - 1; ++w)
    if (w < warp) at += p->sums[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p->off[threadIdx.x * kPer + i] = at;
    at += mine[i];
  }
  if (threadIdx.x == 32 * W - 1) p->off[QD_MAX_SEQS] = at;
  __syncthreads();
}

// A CTA's place in the units: tile group t of a walk (sequence b, kv head h, block of rows r), with
// `left` units of the CTA from there on.
template <int TILE, int W, int BM>
struct Cursor {
  int b, h, r, t, left;
  Walk w;
  int p0, cnt, row0;
  __device__ __forceinline__ void enter(const AttnArgs& a) {
    cnt = tokens_of(a, b, row0, p0);
    w = walk_of<TILE, W, BM>(a, p0, cnt);
  }
  // the first tile group at or behind unit x < off[QD_MAX_SEQS], of n units from x on
  __device__ __forceinline__ void seek(const AttnArgs& a, const Plan<W>& p, int64_t x, int n) {
    b = 0;
#pragma unroll 1
    for (int s = QD_MAX_SEQS / 2; s > 0; s >>= 1)
      if (p.off[b + s] <= x) b += s;
    enter(a);
    const int64_t in = x - p.off[b];
    const int walk = (int)(in / w.len), at = (int)(in - (int64_t)walk * w.len), start = a.whole ? 0 : kStart;
    t = max(at - start, 0);
    left = n - (start + t - at);
    h = walk / w.rb;
    r = walk - h * w.rb;
  }
  __device__ __forceinline__ void next_walk(const AttnArgs& a, const Plan<W>& p) {  // from its last unit
    left -= 1 + (a.whole ? w.len - w.nt : kStart);
    t = 0;
    if (++r < w.rb) return;
    r = 0;
    if (++h < a.c.n_kv) return;
    h = 0;
    do ++b;
    while (b < a.n_seqs && p.off[b] == p.off[b + 1]);
    if (b < a.n_seqs) enter(a);
  }
  __device__ __forceinline__ int last() const { return p0 < 0 ? -1 : p0 + cnt - 1; }  // position of the last row
};

// What a CTA leaves to the join: the walk that began in it and does not end there.
struct Cut {
  int parts, h, r, cnt, row0, pad[3];
};
__host__ __device__ constexpr int part_floats(int bm, int hd) { return bm * (hd + 2); }
constexpr int kMaxCtas = 1024;
constexpr size_t kCutBytes = kMaxCtas * sizeof(Cut);
__device__ __forceinline__ float* part_of(const AttnArgs& a, int bm, int hd, int cta, int slot) {
  return a.ws + kCutBytes / 4 + ((int64_t)cta * 2 + slot) * part_floats(bm, hd);
}
// Row `at` (token, head of the group) of a walk, in an array of rows with this stride.
__device__ __forceinline__ int64_t row_of(const AttnArgs& a, int hd, int64_t stride, int row0, int h, int at) {
  const int token = at / a.group, g = at - token * a.group;
  return (row0 + token) * stride + (int64_t)(h * a.group + g) * hd;
}

// ------------------------------------------------------------------ few rows
// Blocks of 8 or 16 rows, and W warps that walk the positions side by side, each with tiles and a
// ring of its own (no barrier until the walk's end, where the warps' results are joined).  With 8
// rows the two parts of queries and weights are rows 0-7 and 8-15 of one operand, so a product
// serves both.  The operands' columns are free to choose as long as both sides agree: a lane's part
// of a key row is 16 bytes as they lie (its dims of q are the same 16), that of a value row 8 or
// 16, and its outputs are neighbouring dims; nothing is transposed through shared memory, and two
// values of a dim are paired by byte permutations on their way to binary16.
template <int HD, bool R16>
struct Few {
  static constexpr int kW = 4, kStages = HD == 64 ? 3 : 2;
  static constexpr int kTile = 32, kHalf = kTile * HD;  // positions; bytes of keys, of values
  static constexpr int kBm = R16 ? 16 : 8, kCtas = R16 ? 2 : 3;
  uint4 ring[kW][kStages][2][kHalf / 16];  // at a walk's end the slot that was read last: o of the warp's share
  __align__(16) float scales[kW][kStages][2][kTile / 16];
  uint4 q[HD / 16][R16 ? 2 : 1][32];  // the fragments of q's k steps, by lane (16 rows: hi, lo)
  float ml[kW][2][kBm];
  Plan<kW> plan;
};

template <int HD, int FMT, bool R16>
__global__ void __launch_bounds__(Few<HD, R16>::kW * 32, Few<HD, R16>::kCtas) k_paged_few(AttnArgs a) {
  using S = Few<HD, R16>;
  constexpr int W = S::kW, TILE = S::kTile, BM = S::kBm, NB = TILE / 16, NT = TILE / 8, KS = HD / 16, MT = HD / 16;
  constexpr int NR = R16 ? 2 : 1;  // rows of a lane
  constexpr int kLag = S::kStages - 1;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qr = lane >> 2, qc = lane & 3;
  Cut* cut = reinterpret_cast<Cut*>(a.ws) + blockIdx.x;

  pdl_trigger();
  make_plan<TILE, W, BM>(a, &sm.plan);
  const int64_t total = sm.plan.off[QD_MAX_SEQS];
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  per = a.whole ? (per + a.whole - 1) / a.whole * a.whole : max(per, (int64_t)kMinPer);
  const int64_t first = (int64_t)blockIdx.x * per, end = min(first + per, total);
  if (threadIdx.x == 0 && !a.whole) cut->parts = 0;
  if (first >= total) return;
  Cursor<TILE, W, BM> cur, pre;
  cur.seek(a, sm.plan, first, (int)(end - first));
  if (cur.left <= 0) return;
  pre = cur;

  // Copies of this warp's tile at `pre` into the ring, a lane 16 bytes of each 512.  The page of each
  // of its blocks is asked for one step before.
  const uint32_t ring = tc::smem_u32(sm.ring[warp]), scales = tc::smem_u32(sm.scales[warp]);
  // 8 rows of one chunk (keys) and every second of 8 rows (values) without a bank twice; the pattern
  // repeats every 8 rows
  const uint32_t to_k = HD == 64 ? 16 * lane : (lane >> 3) * 128 + (((lane & 7) ^ (4 * (lane >> 3 & 1))) << 4);
  const uint32_t to_v = S::kHalf + (HD == 64 ? (lane >> 3) * 128 + (((lane & 7) ^ (2 * (lane >> 3))) << 4)
                                         : (lane >> 3) * 128 + (((lane & 7) ^ (2 * (lane >> 4))) << 4));
  const uint8_t *from_k = a.c.k + 16 * lane, *from_v = a.c.v + 16 * lane;
  const int own = lane & (NB - 1);  // the block of the tile that the lane looks up, for all, and whose scale it copies
  const float* from_s = lane < NB ? a.c.ks : a.c.vs;
  const int32_t* table;             // the row of the sequence
  int tile, rows, clamp;            // of `pre`; positions from the tile's first one on; the sequence's last block
  int page, in_page;
  auto look = [&] { page = paged::page_of(a.c, table, min(tile * NB + own, clamp), in_page); };
  auto enter_pre = [&] {
    table = paged::table_row(a.c, pre.b);
    tile = pre.w.first_tile + pre.t * W + warp;
    rows = pre.last() + 1 - tile * TILE;
    clamp = max(pre.last(), 0) / QD_KV_BLOCK;
  };
  auto produce = [&](uint32_t s) {  // into slot s, and on to the next
    if (pre.left > 0) {
      const uint32_t mine = page < 0 ? ~0u : (uint32_t)((page * a.c.n_kv + pre.h) * a.c.per_page + in_page);
      const bool all = __all_sync(0xffffffffu, rows >= TILE && mine != ~0u);
      const uint32_t dk = ring + s * (2 * S::kHalf) + to_k, dv = ring + s * (2 * S::kHalf) + to_v, dw = HD == 64 ? dv : dv ^ 64;
      const uint32_t ds = scales + (s * 2 * NB + lane) * 4;
      constexpr int kStep = 16 * HD;  // bytes of a block of keys
      if (all) {
        auto block = [&](auto c) {
          constexpr int k = decltype(c)::value;
          const uint64_t at = (uint64_t)__shfl_sync(0xffffffffu, mine, k) * kStep;
          const uint8_t *fk = from_k + at, *fv = from_v + at;
          cp16<k * kStep, 0>(dk, fk);
          cp16<k * kStep + 512, 512>(dk, fk);
          cp16<k * kStep, 0>(dv, fv);
          cp16<k * kStep + 512, 512>(dw, fv);
          if constexpr (HD == 128) {
            cp16<k * kStep + 1024, 1024>(dk, fk);
            cp16<k * kStep + 1536, 1536>(dk, fk);
            cp16<k * kStep + 1024, 1024>(dv, fv);
            cp16<k * kStep + 1536, 1536>(dw, fv);
          }
        };
        block(std::integral_constant<int, 0>());
        block(std::integral_constant<int, 1>());
        cp4(ds, from_s + mine, lane < 2 * NB);
      } else if (rows > 0) {  // the sequence's last tile, or a block without a page
#pragma unroll 1
        for (int i = 0; i < S::kHalf / 512; ++i) {
          const int byte = 512 * i + 16 * lane;
          const uint32_t at = __shfl_sync(0xffffffffu, mine, 512 * i / kStep);
          const bool live = at != ~0u && byte / HD < rows;
          const uint64_t from = live ? (uint64_t)at * kStep + 512 * i % kStep : 0;
          cp16(dk + 512 * i, from_k + from, live);
          cp16((i & 1 ? dw : dv) + 512 * i, from_v + from, live);
        }
        const bool none = 16 * own >= rows, lost = mine == ~0u;
        cp4(ds, from_s + (none || lost ? 0 : mine), lane < 2 * NB && !none && !lost);
        if (lane < 2 * NB && (none || lost)) (&sm.scales[warp][s][0][0])[lane] = none ? 0.f : __uint_as_float(0x7FC00000u);
      }
      if (pre.t + 1 < pre.w.nt) {
        ++pre.t;
        --pre.left;
        tile += W;
        rows -= W * TILE;
      } else {
        pre.next_walk(a, sm.plan);
        if (pre.left > 0) enter_pre();
      }
      look();
    }
    cp_commit();
  };
  enter_pre();
  look();
#pragma unroll 1
  for (int s = 0; s < kLag; ++s) produce(s);

  float o[MT][NR][4];  // dims HD / 8 qr + 2 i (elements 0, 1), + 1 (2, 3) of rows 8 n + 2 qc, + 1
  float m[NR], l[NR], rs[NR];  // of rows qr + 8 i
  int ev = 0, emax = -1000;
  float down = 1.f;  // 2^-ev
  int lim[NR];               // position of the lane's row, -1: none
  int t_begin, base;         // of the CTA's part of the walk; this warp's first position of the tile
  int top, above, whole_lo, whole_hi;  // tiles with a seen position: above < base <= top; seen by every row: the others
  // a walk's queries: asked for ...
  float4 x[NR][KS];
  auto load_q = [&](const Cursor<TILE, W, BM>& c) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int at = c.r * BM + qr + 8 * i;
      const bool live = at < c.cnt * a.group;
      lim[i] = live && c.p0 >= 0 ? c.p0 + at / a.group : -1;
      const float4* src = reinterpret_cast<const float4*>(a.q + (live ? row_of(a, HD, a.q_stride, c.row0, c.h, at) : 0));
#pragma unroll
      for (int s = 0; s < KS; ++s)  // dims 64 (s / 4) + 16 qc + 4 (s % 4) ..
        x[i][s] = live ? __ldcg(src + (s >> 2) * 16 + 4 * qc + (s & 3)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  // ... and made operands
  auto start_walk = [&](const Cursor<TILE, W, BM>& c) {
    const int low = c.p0 + c.r * BM / a.group;  // position of the block's first row
    top = c.p0 < 0 ? -1 : c.p0 + min(c.cnt - 1, (c.r * BM + BM - 1) / a.group);
    above = a.window > 0 ? low - a.window + 1 - TILE : -TILE;
    whole_lo = a.window > 0 ? top - a.window + 1 : 0;
    whole_hi = low - TILE + 1;
    t_begin = c.t;
    base = (c.w.first_tile + c.t * W + warp) * TILE;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      uint32_t mx = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        x[i][s].x *= a.scale;
        x[i][s].y *= a.scale;
        x[i][s].z *= a.scale;
        x[i][s].w *= a.scale;
        mx = max(mx, abs_max(x[i][s]));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = scale_exp(mx);
      rs[i] = pow2(e);
      const float f = pow2(-e);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (s % W != warp) continue;
        uint32_t hi[2], lo[2];
        split2(x[i][s].x * f, x[i][s].y * f, hi[0], lo[0]);
        split2(x[i][s].z * f, x[i][s].w * f, hi[1], lo[1]);
        if constexpr (R16) {  // hi of rows qr and qr + 8, then lo
          uint32_t* to = reinterpret_cast<uint32_t*>(&sm.q[s][0][lane]) + i;
          to[0] = hi[0];
          to[2] = hi[1];
          to = reinterpret_cast<uint32_t*>(&sm.q[s][R16 ? 1 : 0][lane]) + i;
          to[0] = lo[0];
          to[2] = lo[1];
        } else {  // hi is row qr, lo row qr + 8
          sm.q[s][0][lane] = make_uint4(hi[0], lo[0], hi[1], lo[1]);
        }
      }
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int d = 0; d < MT; ++d)
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][n][e] = 0.f;
    ev = 0;
    emax = -1000;
    down = 1.f;
  };
  load_q(cur);
  start_walk(cur);
  __syncthreads();

  static_assert(BM * HD * 4 <= 2 * S::kHalf, "a share fits a slot");
  auto share = [&](int w, uint32_t slot, int r) { return reinterpret_cast<float*>(sm.ring[w][slot]) + r * HD; };
  for (uint32_t slot = 0;; slot = slot + 1 == S::kStages ? 0 : slot + 1) {
    cp_wait<kLag - 1>();
    __syncwarp();  // every lane's copies have landed, and the slot before this one has been read
    produce(slot == 0 ? S::kStages - 1 : slot - 1);

    if (base <= top && base > above) {
      const unsigned char* kp = reinterpret_cast<const unsigned char*>(sm.ring[warp][slot][0]);
      const unsigned char* vp = reinterpret_cast<const unsigned char*>(sm.ring[warp][slot][1]);
      float ks[NB], vs[NB];
      const float4 scale = *reinterpret_cast<const float4*>(sm.scales[warp][slot]);
      ks[0] = scale.x, ks[1] = scale.y, vs[0] = scale.z, vs[1] = scale.w;
      // ---- scores
      float s[NT][4], lo[R16 ? NT : 1][4];
#pragma unroll
      for (int x = 0; x < HD / 64; ++x) {
        uint4 w[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = 8 * j + qr;
          w[j] = *reinterpret_cast<const uint4*>(
              kp + (HD == 64 ? r * 64 + qc * 16 : r * 128 + (((qc + 4 * x) ^ (4 * (r & 1))) << 4)));
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint4 h = sm.q[4 * x + z][0][lane], g = sm.q[4 * x + z][R16 ? 1 : 0][lane];
          const uint32_t fh[4] = {h.x, h.y, h.z, h.w}, fl[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint32_t b0, b1;
            to_h2x2<FMT>(z == 0 ? w[j].x : z == 1 ? w[j].y : z == 2 ? w[j].z : w[j].w, b0, b1);
            if (x == 0 && z == 0) {
              mma0(s[j], fh, b0, b1);
              if constexpr (R16) mma0(lo[j], fl, b0, b1);
            } else {
              mma(s[j], fh, b0, b1);
              if constexpr (R16) mma(lo[j], fl, b0, b1);
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (R16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] += lo[j][e];
        } else {
          s[j][0] += s[j][2];
          s[j][1] += s[j][3];
        }
      }
      // ---- weights
      const bool edge = base > whole_hi || base < whole_lo;
      // o is in units of 2^ev, so that the tile's scales are 2^-2 to 2 of them: another unit where they are
      // not, at least 2^-60 of the largest (a NaN does not count: there are rows that do not see it)
      float back = 1.f;
      float vtop = fabsf(vs[0]);
#pragma unroll
      for (int k = 1; k < NB; ++k) vtop = fmaxf(vtop, fabsf(vs[k]));
      if (!(vtop * down < 2.f && vtop * down >= 0.25f)) {
        const int etile = vtop <= 3e38f ? max((int)(__float_as_uint(vtop) >> 23) - 127, -100) : -100;
        emax = max(emax, etile);
        const int en = min(max(etile, emax - 60), 126);
        back = pow2(max(min(ev - en, 126), -126));
        ev = en;
        down = pow2(-en);
      }
      float corr[NR], y[NT][2 * NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        // the positions of the tile that the row sees are those from lo to hi
        const int hi = lim[i] - base, lo = a.window > 0 ? hi - a.window + 1 : 0;
        auto sees = [&](int j, int e) { return 8 * j + 2 * qc + e <= hi && 8 * j + 2 * qc + e >= lo; };
        float f[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) f[k] = rs[i] * ks[k];
        if (edge) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              s[j][2 * i + e] = sees(j, e) ? s[j][2 * i + e] * f[j / 2] : -INFINITY;
#pragma unroll
          for (int k = 0; k < NB; ++k) f[k] = 1.f;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < NB; ++k)  // scales are not negative
          mx = fmaxf(mx, f[k] * fmaxf(fmaxf(s[2 * k][2 * i], s[2 * k][2 * i + 1]), fmaxf(s[2 * k + 1][2 * i], s[2 * k + 1][2 * i + 1])));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[i], mx), mu = mn == -INFINITY ? 0.f : mn;
        corr[i] = ex2(m[i] - mu);
        m[i] = mn;
        const float bias = kBias - mu;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p = ex2(fmaf(s[j][2 * i + e], f[j / 2], bias));
            sum += p;
            y[j][2 * i + e] = p * (vs[j / 2] * down);
          }
        if (edge) {  // whatever the scale
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!sees(j, e)) y[j][2 * i + e] = 0.f;
        }
        l[i] = fmaf(l[i], corr[i], sum);
        corr[i] *= back;
      }
      // ---- products with the values
      // transposed, o^T = v^T p^T: a lane's scores are columns of p^T as they stand
      uint32_t ph[NR][NB][2], pl[NR][NB][2];
      float keep[NR][2];  // of rows 8 n + 2 qc, + 1
#pragma unroll
      for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) split2(y[2 * k + x][2 * n], y[2 * k + x][2 * n + 1], ph[n][k][x], pl[n][k][x]);
        keep[n][0] = __shfl_sync(0xffffffffu, corr[n], 8 * qc);
        keep[n][1] = __shfl_sync(0xffffffffu, corr[n], 8 * qc + 4);
      }
      float t[MT][NR][4];
      constexpr int kWords = HD / 32;  // of a lane's part of a value row: 4 dims each
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t v[4][kWords];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = 16 * k + 8 * (x >> 1) + 2 * qc + (x & 1);  // (r >> 1) & 3 == qc
          if constexpr (HD == 64) {
            const uint2 w = *reinterpret_cast<const uint2*>(
                vp + (r >> 1) * 128 + ((((qr >> 1) + 4 * (x & 1)) ^ (2 * qc)) << 4) + 8 * (qr & 1));
            v[x][0] = w.x;
            v[x][1] = w.y;
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(vp + r * 128 + ((qr ^ (2 * qc)) << 4));
            v[x][0] = w.x;
            v[x][1] = w.y;
            v[x][2] = w.z;
            v[x][3] = w.w;
          }
        }
#pragma unroll
        for (int g = 0; g < kWords; ++g) {
          uint32_t d[2][4];  // dims 4 g + 2 i, + 1
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            to_h2x2<FMT>(__byte_perm(v[2 * h][g], v[2 * h + 1][g], 0x5140u), d[0][2 * h], d[0][2 * h + 1]);
            to_h2x2<FMT>(__byte_perm(v[2 * h][g], v[2 * h + 1][g], 0x7362u), d[1][2 * h], d[1][2 * h + 1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              float(&tt)[4] = t[2 * g + i][n];
              if (k == 0) mma0(tt, d[i], pl[n][0][0], pl[n][0][1]);
              else mma(tt, d[i], pl[n][k][0], pl[n][k][1]);
              mma(tt, d[i], ph[n][k][0], ph[n][k][1]);
              if (k == NB - 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[2 * g + i][n][e] = fmaf(o[2 * g + i][n][e], keep[n][e & 1], tt[e]);
              }
            }
        }
      }
    }

    // ---- the end of this CTA's part of the walk
    const bool last = cur.t + 1 == cur.w.nt;
    if (!last && cur.left > 1) {
      ++cur.t;
      --cur.left;
      base += W * TILE;
      continue;
    }
    const bool whole = t_begin == 0 && last;
    __syncwarp();  // every lane has read the slot
    const float unit = pow2(min(max(ev, -126), 127));
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int r = qr + 8 * i;
      if (qc == 0) {
        sm.ml[warp][0][r] = m[i];
        sm.ml[warp][1][r] = l[i];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 0; d < MT; d += 2)
          *reinterpret_cast<float4*>(share(warp, slot, 8 * i + 2 * qc + e) + HD / 8 * qr + 2 * d) =
              make_float4(o[d][i][e] * unit, o[d][i][2 + e] * unit, o[d + 1][i][e] * unit, o[d + 1][i][2 + e] * unit);
    }
    const int done_cnt = cur.cnt, done_r = cur.r, done_h = cur.h, done_row0 = cur.row0;
    const int64_t stop = end - cur.left - cur.t + cur.w.nt - 1;  // the walk's last unit
    cur.next_walk(a, sm.plan);
    const bool more = last && cur.left > 0;
    if (more) load_q(cur);  // on its way meanwhile
    __syncthreads();
    const int live = min(done_cnt * a.group - done_r * BM, BM);
    for (int x = threadIdx.x; x < live * (HD / 4); x += W * 32) {
      const int r = x / (HD / 4), c = x % (HD / 4);
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) mt = fmaxf(mt, sm.ml[w][0][r]);
      float4 ot = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float mw = sm.ml[w][0][r], lw = sm.ml[w][1][r];
        const float f = mw == -INFINITY ? lw : ex2(mw - mt);  // a share without a maximum has l = 0 or NaN
        const float4 ow = *reinterpret_cast<const float4*>(share(w, slot, r) + 4 * c);
        lt = fmaf(lw, f, lt);
        ot.x = fmaf(ow.x, f, ot.x);
        ot.y = fmaf(ow.y, f, ot.y);
        ot.z = fmaf(ow.z, f, ot.z);
        ot.w = fmaf(ow.w, f, ot.w);
      }
      if (whole) {
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        reinterpret_cast<float4*>(a.out + row_of(a, HD, (int64_t)a.n_heads * HD, done_row0, done_h, done_r * BM + r))[c] =
            make_float4(ot.x * inv, ot.y * inv, ot.z * inv, ot.w * inv);
      } else {
        float* part = part_of(a, BM, HD, blockIdx.x, t_begin > 0 ? 0 : 1);
        if (c == 0) {
          part[r] = mt;
          part[BM + r] = lt;
        }
        reinterpret_cast<float4*>(part + 2 * BM + r * HD)[c] = ot;
      }
    }
    if (!whole && t_begin == 0 && threadIdx.x == 0) {
      cut->parts = (int)(stop / per) - (int)blockIdx.x + 1;
      cut->h = done_h;
      cut->r = done_r;
      cut->cnt = done_cnt;
      cut->row0 = done_row0;
    }
    if (more) start_walk(cur);
    __syncthreads();  // every share has been read, and q stands
    if (!more) break;
  }
  cp_wait<0>();
}

// The parts of a cut walk, in the CTAs' order: a block to a row of the walk that CTA blockIdx.x began.
constexpr int kJoinThreads = 128;
template <int HD, int BM>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(AttnArgs a) {
  constexpr int kLanes = HD / 4, kGroups = kJoinThreads / kLanes;
  __shared__ float s_w[kMaxCtas];
  __shared__ float s_red[kJoinThreads / 32];
  __shared__ float4 s_o[kGroups][kLanes];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();  // in every CTA: the end of this kernel is the end of both
  const Cut* cut = reinterpret_cast<const Cut*>(a.ws) + blockIdx.x;
  const int n = __ldcg(&cut->parts), r = blockIdx.y;
  if (n == 0) return;
  const int at = __ldcg(&cut->r) * BM + r;
  if (at >= __ldcg(&cut->cnt) * a.group) return;
  auto part = [&](int i) { return part_of(a, BM, HD, blockIdx.x + i, i == 0 ? 1 : 0); };
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < n; i += kJoinThreads) {
    s_w[i] = __ldcg(part(i) + r);
    mx = fmaxf(mx, s_w[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) s_red[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, s_red[w]);
  __syncthreads();
  float l = 0.f;
  for (int i = threadIdx.x; i < n; i += kJoinThreads) {
    const float lp = __ldcg(part(i) + BM + r);
    s_w[i] = s_w[i] == -INFINITY ? lp : ex2(s_w[i] - mx);  // a part without a maximum has l = 0 or NaN
    l = fmaf(lp, s_w[i], l);
  }
  l = warp_sum(l);
  if (lane == 0) s_red[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) l += s_red[w];
  const int g = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = g; i < n; i += kGroups) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(part(i) + 2 * BM + r * HD) + c);
    const float w = s_w[i];
    o.x = fmaf(x.x, w, o.x);
    o.y = fmaf(x.y, w, o.y);
    o.z = fmaf(x.z, w, o.z);
    o.w = fmaf(x.w, w, o.w);
  }
  s_o[g][c] = o;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) {
    const float4 x = s_o[i][c];
    o.x += x.x;
    o.y += x.y;
    o.z += x.z;
    o.w += x.w;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<float4*>(a.out + row_of(a, HD, (int64_t)a.n_heads * HD, __ldcg(&cut->row0), __ldcg(&cut->h), at))[c] =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

// ------------------------------------------------------------------ host
inline bool attn_shape_ok(const qd_paged_kv* kv, int n_heads, int n_tokens, int n_seqs) {
  return paged::cache_status(kv, n_seqs) == QD_OK && n_heads >= 1 && n_heads % kv->n_kv_heads == 0 &&
         n_heads / kv->n_kv_heads <= 16 && n_tokens >= 1 && n_tokens <= QD_MAX_GEMM_TOKENS;
}
inline bool rows16(int group, int n_tokens, int n_seqs) { return group > 8 || n_tokens > n_seqs; }

// CTAs of a call: what fits the device at once, and no more than there can be units for.
inline int few_ctas(const Cache& c, int tile, int w, int bm, int per_sm, int group, int n_tokens, int n_seqs) {
  const int64_t walks = ((int64_t)n_tokens * group / bm + std::min(n_tokens, n_seqs)) * c.n_kv;
  const int64_t most = (c.capacity + tile * w - 1) / (tile * w) + kStart;  // units of a walk
  const int64_t ctas = std::min({(int64_t)attn_sm_count() * per_sm, (int64_t)kMaxCtas, (walks * most + kMinPer - 1) / kMinPer});
  return (int)std::max<int64_t>(ctas, 1);
}

template <int HD, int FMT, bool R16>
qd_status launch_few(AttnArgs a, cudaStream_t st) {
  using S = Few<HD, R16>;
  static std::atomic<bool> done[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QD_ERR_CUDA;
  const auto kern = k_paged_few<HD, FMT, R16>;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S)) != cudaSuccess)
      return QD_ERR_CUDA;
    done[dev] = true;
  }
  const int most = (a.c.capacity + S::kTile * S::kW - 1) / (S::kTile * S::kW);
  a.whole = most <= kWholeUnits ? most : 0;
  const int ctas = few_ctas(a.c, S::kTile, S::kW, S::kBm, S::kCtas, a.group, a.n_tokens, a.n_seqs);
  kern<<<ctas, S::kW * 32, sizeof(S), st>>>(a);
  const qd_status s = launch_status();
  if (s != QD_OK || a.whole) return s;
  return launch_k(k_paged_join<HD, S::kBm>, dim3((unsigned)ctas, S::kBm), dim3(kJoinThreads), 0, st, true, a);
}

template <int HD, int FMT>
qd_status launch_attn(const AttnArgs& a, cudaStream_t st) {
  return rows16(a.group, a.n_tokens, a.n_seqs) ? launch_few<HD, FMT, true>(a, st) : launch_few<HD, FMT, false>(a, st);
}

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

size_t qd_paged_attn_workspace(const qd_paged_kv* kv, int n_heads, int n_tokens, int n_seqs) {
  if (!attn_shape_ok(kv, n_heads, n_tokens, n_seqs)) return 0;
  const int64_t ctas = std::min(attn_sm_count() * 4, kMaxCtas);  // whatever the call: it serves them all
  return kCutBytes + (size_t)ctas * 2 * part_floats(16, kv->head_dim) * sizeof(float);
}

qd_status qd_paged_attn(const qd_paged_kv* kv, const float* q, int64_t q_stride, float* out, int n_heads, int n_tokens,
                        const int32_t* row_start, const int32_t* pos, int n_seqs, float scale, int window,
                        void* workspace, size_t workspace_bytes, qd_stream_t stream) {
  if (!q || !out || !row_start || !pos || !workspace || window < 0 || !std::isfinite(scale)) return QD_ERR_INVALID_ARG;
  const qd_status r = paged::cache_status(kv, n_seqs);
  if (r != QD_OK) return r;
  const size_t need = qd_paged_attn_workspace(kv, n_heads, n_tokens, n_seqs);
  if (!need) return QD_ERR_SHAPE;
  if (n_tokens > 1 && q_stride < (int64_t)n_heads * kv->head_dim) return QD_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned4(row_start) || !aligned4(pos) ||
      (n_tokens > 1 && q_stride % 4))
    return QD_ERR_ALIGN;
  if (workspace_bytes < need) return QD_ERR_NOMEM;
  AttnArgs a = {};
  a.c = paged::cache_of(kv);
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.n_heads = n_heads;
  a.n_tokens = n_tokens;
  a.n_seqs = n_seqs;
  a.group = n_heads / kv->n_kv_heads;
  a.row_start = row_start;
  a.pos = pos;
  a.scale = scale * 1.4426950408889634f;
  a.window = window;
  a.max_rows = 1 << 30;
  a.ws = static_cast<float*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (kv->head_dim == 64)
    return kv->fmt == QD_KV_I8 ? launch_attn<64, QD_KV_I8>(a, st) : launch_attn<64, QD_KV_E4M3>(a, st);
  return kv->fmt == QD_KV_I8 ? launch_attn<128, QD_KV_I8>(a, st) : launch_attn<128, QD_KV_E4M3>(a, st);
}

}  // extern "C"
