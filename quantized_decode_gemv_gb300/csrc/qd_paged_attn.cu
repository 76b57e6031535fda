// Causal attention of packed rows over the pages of an 8-bit cache:
//   o = sum_j softmax_j(scale q . k_j) v_j,  k_j = code * scale of its block, over the positions
// j = 0 .. p of a row at position p (the last `window` of them with a window).
//
// The rows that share a kv head (tokens x query heads of the group) walk its positions together
// with an online softmax: s = q k^T and o += p v are matrix products with f32 accumulators.  Codes
// of 8 bits are exact in binary16, so they enter the products as they are; a block's scale of keys
// multiplies its scores, that of values its weights.  Outputs are f32 and meant to be as exact as f32
// arithmetic, so queries and weights times scales enter in two binary16 parts, hi = rn(x), lo = rn(x - hi), at a
// power of two that puts the largest of a row at 2^14 to 2^15 (2^15.1 for weights): what is 2^-15 of that or more
// keeps 22 bits, what is less is 2^-38 of it off.  The matrix units
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
// The kernel for few rows.  kMinPer 2 against 1, one sequence, in us: 3 heads of 2000 positions 8.6 and 8.2, one head of
// 16000 10.7 and 11.9; against 4: 8.6 and 10.6, 10.7 and 11.4.  kWholeUnits 4 against 1: 3 heads of 500 positions 8.1
// and 8.5, 16 x 32 heads of 500 at most 15.4 and 14.1; against 16: 3 heads of 2000 8.6 and 20.0.
constexpr int kStart = 1;       // what the start of a walk costs, in units
constexpr int kMinPer = 2;      // units of a CTA at least
constexpr int kWholeUnits = 4;  // where the table has room for at most so many units, no walk is cut

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

// o is held in units of 2^ev of its row, ev the floor of the running maximum of score + log2 scale over the positions
// that the row sees, less that of the scores, so that the largest weight times scale is 2^14 to 2^15.1 times the unit,
// whatever a block weighs that the row does not see, or that has a large scale and no weight.
__device__ __forceinline__ float log2_scale(float s) {  // log2 or up to 0.09 less; finite for any s
  return fmaf((float)__float_as_int(s), 0x1p-23f, -127.f);
}
// The next ev for that difference; back: what o in the old unit is multiplied by.
__device__ __forceinline__ void next_unit(float n, int& ev, float& back, float& down) {
  const int en = min(max(__float2int_rd(n), -100), 126);
  back = pow2(max(min(ev - en, 126), -126));
  down = pow2(-en);
  ev = en;
}
// Scores from here on have steps of 2^-2 and more.  A fused product and difference would leave the rounding of the maximum
// in the largest weight, which is to end at 2^14, and so would the sum of the maximum and 14: both are rounded alike, and
// the largest weight is 1.
constexpr float kHuge = 0x1p22f;
__device__ __forceinline__ float bias_of(float m, bool huge) { return huge ? -m : kBias - m; }
// A share of a row, as it is joined with others: the maximum score m, the sum l of the weights, and o scaled by
// down_of(l), so that it is no larger than the row's largest value (where these are near f32's largest, their sum has
// no place in it).  With weights ex2(m - the largest m), o of several is sum of w up_of(l) o, times down_of(sum of w l).
__device__ __forceinline__ float down_of(float l) { return __int_as_float((253 - (__float_as_int(l) >> 23)) << 23); }
__device__ __forceinline__ float up_of(float l) { return __int_as_float(((__float_as_int(l) >> 23) + 1) << 23); }
// What makes o the mean.
__device__ __forceinline__ float inv_of(float l) { return l == 0.f ? 0.f : 1.f / (l * down_of(l)); }
// s down, not over the largest finite value: a scale that the row hardly sees may be 2^100 units; NaN stays
__device__ __forceinline__ float in_units(float s, float down) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(s * down), "f"(3e38f));
  return y;
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

// Every block of rows walks what any row of its sequence sees, and leaves out the products of what its own do not (8/1
// heads of 64, 1000 tokens, a window of 16: 21 us).
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
// values of a dim are paired by byte permutations on their way to binary16 (2.5 instructions a pair of keys,
// 3 of values).
// What bounds it: the dependent chain of a tile (copies, scores, maximum, weights, products), which the 8 or 12 warps
// that an SM's registers hold do not hide.  A warp takes about 480 instructions for 4 KB of the cache (176 turn codes into
// operands, 32 are products; starts and joins among them), of which an SM issues 1.5 to 2 of 4 a cycle, where HBM brings
// 4 KB in 174 cycles.  The kernels of head dimension 128 spill (76 to 92 bytes a thread with 8 rows, 164 to 212 with 16).
// 100 sequences of 32/8 heads of 128, 4000 positions on average: 166 us (floor 123); 131000 positions of one: 59 (40);
// 16 of 32/32 heads of 64, 2000 on average: 40 (20, and 8 of the starts and the join).  Against, at the time: tiles of 4 KB
// at head dimension 128 178 us instead of 166, tiles of 8 KB at 64 46 instead of 40; four CTAs of 128 registers a
// thread 253 (more spills) and 44; CTAs of two warps 227 and 39; q's fragments in registers 171 and 38;
// o = p v instead of its transpose, where both parts of a weight have accumulators of their own, 171 and 41;
// kStart 3 166 and 40.5, 5 169 and 43.
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
  float n[NR];
  int ev[NR];
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
      m[i] = n[i] = -INFINITY;
      ev[i] = 0;
      l[i] = 0.f;
    }
#pragma unroll
    for (int d = 0; d < MT; ++d)
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][n][e] = 0.f;
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
      float lgv[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) lgv[k] = log2_scale(vs[k]);
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
        float mk[NB], mn = m[i];  // the blocks' maxima
#pragma unroll
        for (int k = 0; k < NB; ++k) {  // scales are not negative
          mk[k] = f[k] * fmaxf(fmaxf(s[2 * k][2 * i], s[2 * k][2 * i + 1]), fmaxf(s[2 * k + 1][2 * i], s[2 * k + 1][2 * i + 1]));
          mk[k] = fmaxf(mk[k], __shfl_xor_sync(0xffffffffu, mk[k], 1));
          mk[k] = fmaxf(mk[k], __shfl_xor_sync(0xffffffffu, mk[k], 2));
          mn = fmaxf(mn, mk[k]);
        }
        const float mu = mn == -INFINITY ? 0.f : mn;
        corr[i] = ex2(m[i] - mu);
        n[i] += m[i] - mu;
        m[i] = mn;
#pragma unroll
        for (int k = 0; k < NB; ++k) n[i] = fmaxf(n[i], (mk[k] - mu) + lgv[k]);
        float back, down, vu[NB];
        next_unit(n[i], ev[i], back, down);
        const bool huge = fabsf(mu) >= kHuge;
        if (huge) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[j][2 * i + e] *= f[j / 2];
#pragma unroll
          for (int k = 0; k < NB; ++k) f[k] = 1.f;
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) vu[k] = in_units(vs[k], down);
        const float bias = bias_of(mu, huge);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p = ex2(fmaf(s[j][2 * i + e], f[j / 2], bias));
            sum += p;
            y[j][2 * i + e] = p * vu[j / 2];
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
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const float unit = pow2(ev[i]), norm = down_of(l[i]);
      const int r = qr + 8 * i;
      if (qc == 0) {
        sm.ml[warp][0][r] = m[i];
        sm.ml[warp][1][r] = l[i];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float u = __shfl_sync(0xffffffffu, unit, 8 * qc + 4 * e), f = __shfl_sync(0xffffffffu, norm, 8 * qc + 4 * e);
#pragma unroll
        for (int d = 0; d < MT; d += 2)
          *reinterpret_cast<float4*>(share(warp, slot, 8 * i + 2 * qc + e) + HD / 8 * qr + 2 * d) =
              make_float4(o[d][i][e] * f * u, o[d][i][2 + e] * f * u, o[d + 1][i][e] * f * u, o[d + 1][i][2 + e] * f * u);
      }
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
      float f[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float mw = sm.ml[w][0][r], lw = sm.ml[w][1][r];
        f[w] = mw == -INFINITY ? lw : ex2(mw - mt);  // a share without a maximum has l = 0 or NaN
        lt = fmaf(lw, f[w], lt);
        f[w] *= up_of(lw);
      }
      const float norm = down_of(lt);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float4 ow = *reinterpret_cast<const float4*>(share(w, slot, r) + 4 * c);
        f[w] *= norm;
        ot.x = fmaf(ow.x, f[w], ot.x);
        ot.y = fmaf(ow.y, f[w], ot.y);
        ot.z = fmaf(ow.z, f[w], ot.z);
        ot.w = fmaf(ow.w, f[w], ot.w);
      }
      if (whole) {
        const float inv = inv_of(lt);
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
    const float f = s_w[i] == -INFINITY ? lp : ex2(s_w[i] - mx);  // a part without a maximum has l = 0 or NaN
    l = fmaf(lp, f, l);
    s_w[i] = f * up_of(lp);
  }
  l = warp_sum(l);
  if (lane == 0) s_red[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) l += s_red[w];
  const float norm = down_of(l);
  const int g = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = g; i < n; i += kGroups) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(part(i) + 2 * BM + r * HD) + c);
    const float w = s_w[i] * norm;
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
  const float inv = inv_of(l);
  reinterpret_cast<float4*>(a.out + row_of(a, HD, (int64_t)a.n_heads * HD, __ldcg(&cut->row0), __ldcg(&cut->h), at))[c] =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

// ------------------------------------------------------------------ many rows
// Sequences of more rows than kFewRows: blocks of 128 on the 5th-generation tensor cores, two threads to a
// row.  All threads convert a tile's codes (64 positions) to binary16 operands in shared memory, 8 x 8 core
// matrices of 128 bytes: row r, 16-byte chunk c at core_off(r, c).  One thread issues s = q k^T (tcgen05.mma,
// M = 128, N = 64, q's parts in shared memory) into one of two score buffers in tensor memory; a row's threads
// read half of its scores each, exchange their maxima, read the scores again and write the weights' parts over
// them as the A operand of o = p v (V as it lies, [position][dim], is the transposed B operand); each adds half
// of the tile's dims to its own registers, rounded.  The next tile's keys are converted and its scores issued
// under the products with the values, its values converted and the sums made under those scores; two CTAs to an
// SM fill what is left.  The blocks of all walks, as long as each block's last row sees, are listed by a kernel
// of one CTA and taken whole or cut evenly over the CTAs, in heads, sequences and blocks in turn.
// What bounds it: the latency of a tile's chain between its three barriers (1.3 of 4 instructions a cycle; a tile
// of 128 rows takes a CTA 3.5 us alone on an SM; 112 bytes a thread are spilled at head dimension 128).  8 heads of 128,
// 1024 x 4 rows, 2040 positions: 137 to 142 us, of which the list 5 and the join that finds nothing 3 (floor 13: the
// products once); in copies, of 136 us then, without the conversions 99 us, without the products too 76, with a quarter of
// the sums too 67.  Against the same 136: walks cut 151 us, 17 of them the join; the next loads before the proxy fences 144;
// four threads to a row, of 64 registers, 167; the values' codes through shared memory 143; blocks of 16 rows 277.  A
// row's units of its own cost 5 us with the bounds of the block's rows in registers, none with them in the segment.
constexpr int kManyThreads = 256, kManyTile = 64, kManyBm = 128;
// 8 heads of 128, 16000 positions, few against many rows: 16 sequences of 32 rows 290 and 431 us, 8 of 64 288 and
// 246, 8 of 80 346 and 251, 8 of 120 547 and 262.
constexpr int kFewRows = 48;
constexpr int kManyStart = 2, kManyMinPer = 4;  // what a walk's start costs, in tiles; tiles of a CTA at least
constexpr int kManyJoin = 4;                     // what the join costs, in tiles
constexpr int kListThreads = 1024;

// A block of rows that a walk stands for, with the units (tiles, and kManyStart) of those before it.
struct Block {
  int off, seq, r, first_tile, nt, pad[3];
};
struct ManyHead {
  int blocks, units;  // of a head
  int whole;          // 1: no walk is cut
  int pad[5];
};
// The workspace: what both kernels' cuts need, the list, the parts.
inline int most_blocks(int group, int n_tokens, int n_seqs) {
  return (int)((int64_t)n_tokens * group / kManyBm) + std::min(n_tokens, n_seqs);
}
inline size_t list_bytes(int group, int n_tokens, int n_seqs) {
  return sizeof(ManyHead) + (size_t)most_blocks(group, n_tokens, n_seqs) * sizeof(Block);
}
struct ManyArgs {
  AttnArgs a;
  int min_rows;     // sequences of fewer are the other kernel's
  int ctas;
  int most;         // blocks that the list has room for: all of them where row_start ascends
  ManyHead* head;   // the list behind it
  Cut* cuts;
  float* parts;
};

__global__ void __launch_bounds__(kListThreads) k_paged_list(ManyArgs m) {
  __shared__ int s_start[QD_MAX_SEQS + 1], s_sum[kListThreads / 32];
  __shared__ int s_base, s_longest;
  const AttnArgs& a = m.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto scan = [&](int v, int& sum) {  // exclusive over the CTA
    int upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll 8
    for (int w = 0; w < kListThreads / 32; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    __syncthreads();
    sum = all;
    return before + upto - v;
  };
  int n = 0, all;
  if (tid < a.n_seqs) {
    int row0, p0;
    const int64_t rows = (int64_t)tokens_of(a, tid, row0, p0) * a.group;
    if (rows >= m.min_rows) n = (int)((rows + kManyBm - 1) / kManyBm);
  }
  const int at = scan(n, all);
  if (tid <= QD_MAX_SEQS) s_start[tid] = at;  // those behind the last sequence: all of them
  if (tid == 0) s_base = s_longest = 0;
  __syncthreads();
  Block* list = reinterpret_cast<Block*>(m.head + 1);
  all = min(all, m.most);
  for (int i0 = 0; i0 < all; i0 += kListThreads) {
    const int i = i0 + tid;
    Block b = {};
    int len = 0, sum;
    if (i < all) {
      int q = 0;
#pragma unroll 1
      for (int s = QD_MAX_SEQS / 2; s > 0; s >>= 1)
        if (s_start[q + s] <= i) q += s;
      int row0, p0;
      const int t = tokens_of(a, q, row0, p0);
      b.seq = q;
      b.r = i - s_start[q];
      b.nt = 1;
      if (p0 >= 0) {
        const int low = p0 + b.r * kManyBm / a.group, top = p0 + min(t - 1, (b.r * kManyBm + kManyBm - 1) / a.group);
        b.first_tile = a.window > 0 ? max(low - a.window + 1, 0) / kManyTile : 0;
        b.nt = top / kManyTile - b.first_tile + 1;
      }
      len = b.nt + kManyStart;
      atomicMax(&s_longest, len);
    }
    const int before = scan(len, sum);
    b.off = s_base + before;
    if (i < all) list[i] = b;
    __syncthreads();
    if (tid == 0) s_base += sum;
    __syncthreads();
  }
  if (tid == 0) {
    m.head->blocks = all;
    m.head->units = s_base;
    // Cut walks are even, but their parts are written, read and joined (66 KB each); whole ones cost nothing
    // more where there are enough of them and none is much longer than a CTA's share.
    const int64_t walks = (int64_t)all * a.c.n_kv, share = ((int64_t)s_base * a.c.n_kv + m.ctas - 1) / m.ctas;
    m.head->whole = walks >= m.ctas / 2 && (walks + m.ctas - 1) / m.ctas * s_longest <= share * 8 / 5 + kManyJoin;
  }
}

__device__ __forceinline__ bool elect_one() {  // one lane of the (whole) calling warp
  uint32_t p;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(p));
  return p != 0;
}
// 16 consecutive 32-bit columns of this thread's tensor-memory lane read, 8 written
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int HD>
__device__ __forceinline__ uint32_t core_off(int r, int c) {  // in bytes
  return (uint32_t)(((r >> 3) * (HD / 8) + c) * 128 + (r & 7) * 16);
}

// A CTA's part of a walk: n tiles from t0 on.
struct Segment {
  int h, r, cnt, row0, p0, seq, first_tile, nt, t0, n;
  int low, top;  // positions of the block's first and last row
};
template <int HD>
struct Many {
  uint4 q[2][kManyBm * HD / 8];    // hi, lo
  uint4 k[kManyTile * HD / 8], v[kManyTile * HD / 8];
  __align__(16) float scales[2][3][4];  // of every second tile's blocks: keys, values, log2_scale of those
  uint32_t place[2][4];            // of every second tile: its blocks in the cache, kNoPage
  float2 ex[2][kManyBm];           // what a row's threads tell each other
  unsigned long long mbar[2];      // scores, products
  int whole;
  long long unit;                  // of the next segment: its place in all units (of walks where they are whole),
  int left, in, block, head;       // the CTA's units from there on, its place in the walk, the walk
  uint32_t tmem;
  Segment seg;
};

template <int HD, int FMT>
__global__ void __launch_bounds__(kManyThreads, 2) k_paged_many(ManyArgs ma) {
  using S = Many<HD>;
  constexpr int T = kManyTile, BM = kManyBm, ND = HD / 2, kCols = 256;
  constexpr uint32_t kColsO = 2 * T;
  constexpr uint32_t kIdescS = tc::idesc_f16(BM, T), kIdescO = tc::idesc_f16(BM, HD) | (1u << 16);  // B: N contiguous
  static_assert(2 * T + HD <= kCols, "tensor memory of half an SM");
  constexpr int kPer = HD / 64;  // 16-byte pieces of a tile's keys (values) to a thread
  extern __shared__ __align__(128) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const AttnArgs& a = ma.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lrow = tid & 127, half = tid >> 7;
  const int uwarp = __shfl_sync(0xffffffffu, warp, 0);  // known to be the warp's: descriptors stay in uniform registers

  pdl_trigger();
  int64_t per;
  {
    const int n_blocks = ma.head->blocks, head_units = ma.head->units;
    const int64_t total = (int64_t)head_units * a.c.n_kv;
    per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kManyMinPer);
    const int64_t first = (int64_t)blockIdx.x * per;
    if (tid == 0) ma.cuts[blockIdx.x].parts = 0;
    const int whole = ma.head->whole;
    if (whole ? (int64_t)blockIdx.x >= (int64_t)n_blocks * a.c.n_kv : first >= total) return;
    if (tid == 0) sm.whole = whole;
    if (tid == 0 && whole) sm.unit = blockIdx.x;
    if (tid == 0 && !whole) {
      const Block* list = reinterpret_cast<const Block*>(ma.head + 1);
      sm.unit = first;
      sm.left = (int)min(per, total - first);
      sm.head = (int)(first / head_units);
      const int in = (int)(first - (int64_t)sm.head * head_units);
      int lo = 0, hi = n_blocks;  // the last block with off <= in
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (list[mid].off <= in) lo = mid;
        else hi = mid;
      }
      sm.block = lo;
      sm.in = in - list[lo].off;
    }
  }
  // One thread: the part of the walk (head, block) from unit `in` on into sm.seg, and on to the next; n = 0: none left.
  auto set_segment = [&](Segment& g) {
    g.low = g.top = -1;  // out of range: no row sees a position
    if (g.p0 >= 0) {
      g.low = g.p0 + g.r * BM / a.group;
      g.top = g.p0 + min(g.cnt - 1, (g.r * BM + BM - 1) / a.group);
    }
    sm.seg = g;
  };
  auto next_segment = [&] {
    const Block* list = reinterpret_cast<const Block*>(ma.head + 1);
    Segment g = {};
    if (sm.whole) {  // every gridDim.x-th walk, the last blocks of a sequence, which see most, first
      const int n_blocks = ma.head->blocks;
      if (sm.unit < (int64_t)n_blocks * a.c.n_kv) {
        const Block b = list[n_blocks - 1 - (int)(sm.unit / a.c.n_kv)];
        g.h = (int)(sm.unit % a.c.n_kv);
        g.r = b.r;
        g.seq = b.seq;
        g.first_tile = b.first_tile;
        g.n = g.nt = b.nt;
        g.cnt = tokens_of(a, b.seq, g.row0, g.p0);
        sm.unit += gridDim.x;
      }
      set_segment(g);
      return;
    }
    while (g.n <= 0 && sm.left > 0) {
      const Block b = list[sm.block];
      const int in = sm.in, left = sm.left;
      g.t0 = max(in - kManyStart, 0);
      g.n = min(b.nt - g.t0, left - (g.t0 + kManyStart - in));
      g.h = sm.head;
      g.r = b.r;
      g.seq = b.seq;
      g.first_tile = b.first_tile;
      g.nt = b.nt;
      g.cnt = tokens_of(a, b.seq, g.row0, g.p0);
      if (g.n > 0 && g.t0 == 0 && g.n < g.nt) {  // goes on in the next CTAs
        Cut* cut = ma.cuts + blockIdx.x;
        cut->parts = (int)((sm.unit - in + kManyStart + g.nt - 1) / per) - (int)blockIdx.x + 1;
        cut->h = g.h;
        cut->r = g.r;
        cut->cnt = g.cnt;
        cut->row0 = g.row0;
      }
      const int rest = kManyStart + b.nt - in;  // units of the walk from here on
      sm.unit += rest;
      sm.left = left - rest;
      sm.in = 0;
      if (++sm.block == ma.head->blocks) {
        sm.block = 0;
        ++sm.head;
      }
    }
    set_segment(g);
  };

  const uint32_t mb_s = tc::smem_u32(&sm.mbar[0]), mb_o = tc::smem_u32(&sm.mbar[1]);
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&sm.tmem)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    tc::mbar_init(mb_s, 1);
    tc::mbar_init(mb_o, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    next_segment();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = sm.tmem, mine = tm + ((uint32_t)(32 * (warp & 3)) << 16);  // this warp's lanes

  // A warp takes 8 rows of a tile and 64 dims: 8 rows of one chunk of 8 dims are a core matrix.
  const int trow = (warp >> (kPer - 1)) * 8 + (lane & 7);            // row of the first piece; the second: 32 rows on
  const int piece = (lane >> 3) + (kPer == 2 ? 4 * (warp & 1) : 0);  // of 16 dims
  constexpr uint32_t kNoPage = ~0u;
  const uint32_t in_block = (trow & 15) * HD + 16 * piece;
  uint4 kc[kPer], vc[kPer];
  int head = 0, last = -1;  // of the walk: its kv head, the sequence's last position
  // Eight threads: where the blocks of a tile are, two tiles before the tile, and their scales, one before
  // (a thread a block and K or V).
  const int32_t* table = nullptr;
  uint32_t my_place = kNoPage;
  float scale = 0.f;
  auto look = [&](int tile) {
    if (tid >= 8) return;
    int in_page;
    const int page = paged::page_of(a.c, table, min(tile * 4 + (tid & 3), max(last, 0) / QD_KV_BLOCK), in_page);
    my_place = page < 0 ? kNoPage : (uint32_t)((page * a.c.n_kv + head) * a.c.per_page + in_page);
  };
  auto tell = [&](int tile) {
    if (tid < 4) sm.place[tile & 1][tid] = my_place;
  };
  auto load_scale = [&](int tile) {  // looked up before
    if (tid >= 8) return;
    scale = (tile * 4 + (tid & 3)) * QD_KV_BLOCK > last ? 0.f
            : my_place == kNoPage                       ? __uint_as_float(0x7FC00000u)
                                                        : __ldg((tid < 4 ? a.c.ks : a.c.vs) + my_place);
  };
  auto put_scale = [&](int slot) {
    sm.scales[slot][tid >> 2][tid & 3] = scale;
    if (tid >= 4) sm.scales[slot][2][tid & 3] = log2_scale(scale);
  };
  auto load_codes = [&](const uint8_t* codes, int tile, uint4 (&c)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t at = sm.place[tile & 1][(trow >> 4) + 2 * i];
      const bool live = at != kNoPage && tile * T + trow + 32 * i <= last;
      const uint8_t* from = codes + ((uint64_t)at * (16 * HD) + in_block);
      asm volatile(  // zeros behind the sequence's end
          "{\n"
          ".reg .pred p;\n"
          "setp.ne.u32 p, %5, 0;\n"
          "mov.u32 %0, 0;\n"
          "mov.u32 %1, 0;\n"
          "mov.u32 %2, 0;\n"
          "mov.u32 %3, 0;\n"
          "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n"
          "}\n"
          : "=&r"(c[i].x), "=&r"(c[i].y), "=&r"(c[i].z), "=&r"(c[i].w)
          : "l"(from), "r"((uint32_t)live));
    }
  };
  auto convert = [&](const uint4 (&c)[kPer], uint4* to) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      uint4 x, y;
      to_h2x2<FMT>(c[i].x, x.x, x.y);
      to_h2x2<FMT>(c[i].y, x.z, x.w);
      to_h2x2<FMT>(c[i].z, y.x, y.y);
      to_h2x2<FMT>(c[i].w, y.z, y.w);
      to[core_off<HD>(trow + 32 * i, 2 * piece) / 16] = x;
      to[core_off<HD>(trow + 32 * i, 2 * piece + 1) / 16] = y;
    }
  };
  // One thread: s = q k^T into score buffer b, lo of q first (what is cut off there does not count)
  auto issue_s = [&](int b) {
    tc::fence_after_sync();
#pragma unroll
    for (int part = 1; part >= 0; --part)
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks)
        tc::mma_f16_ss(tm + T * b, tc::smem_desc(tc::smem_u32(sm.q[part]) + 256 * ks, 128, HD * 16),
                       tc::smem_desc(tc::smem_u32(sm.k) + 256 * ks, 128, HD * 16), kIdescS, part == 0 || ks > 0);
    tc::mma_commit(mb_s);
  };
  auto issue_o = [&](int b) {
    tc::fence_after_sync();
#pragma unroll
    for (int part = 1; part >= 0; --part)
#pragma unroll
      for (int kk = 0; kk < T / 16; ++kk)  // 16 positions: 8 columns of p, two rows of core matrices of v
        tc::mma_f16_ts(tm + kColsO, tm + T * b + 16 * kk + 8 * part,
                       tc::smem_desc(tc::smem_u32(sm.v) + HD * 32 * kk, HD * 16, 128), kIdescO, part == 0 || kk > 0);
    tc::mma_commit(mb_o);
  };

  bool lost = false;  // a wait has run out: the rows of the walk are NaN
  uint32_t it = 0;    // tiles of this CTA so far
  while (sm.seg.n > 0) {
    float o[ND], m = -INFINITY, n = -INFINITY, l = 0.f, rs;
    int ev = 0, lim, tile, stop;
    {
      const Segment& g = sm.seg;
      head = g.h;
      last = g.p0 < 0 ? -1 : g.p0 + g.cnt - 1;
      table = paged::table_row(a.c, g.seq);
      tile = g.first_tile + g.t0;
      stop = tile + g.n;
      look(tile);
      tell(tile);
      load_scale(tile);
      // ---- queries
      const int row = g.r * BM + lrow;
      const bool live = row < g.cnt * a.group;
      lim = live && g.p0 >= 0 ? g.p0 + row / a.group : -1;
      const float4* src = reinterpret_cast<const float4*>(a.q + (live ? row_of(a, HD, a.q_stride, g.row0, g.h, row) : 0) + half * ND);
      uint32_t mx = 0;
#pragma unroll
      for (int d = 0; d < ND; d += 4) {
        const float4 x = live ? __ldcg(src + d / 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        o[d] = x.x * a.scale;
        o[d + 1] = x.y * a.scale;
        o[d + 2] = x.z * a.scale;
        o[d + 3] = x.w * a.scale;
        mx = max(mx, abs_max(make_float4(o[d], o[d + 1], o[d + 2], o[d + 3])));
      }
      sm.ex[half][lrow].x = __uint_as_float(mx);
      __syncthreads();
      load_codes(a.c.k, tile, kc);
      load_codes(a.c.v, tile, vc);
      look(tile + 1);
      tell(tile + 1);
      const int e = scale_exp(max(mx, __float_as_uint(sm.ex[half ^ 1][lrow].x)));
      rs = pow2(e);
      const float f = pow2(-e);
#pragma unroll
      for (int c = 0; c < ND / 8; ++c) {
        uint4 hi, lo;
        split2(o[8 * c] * f, o[8 * c + 1] * f, hi.x, lo.x);
        split2(o[8 * c + 2] * f, o[8 * c + 3] * f, hi.y, lo.y);
        split2(o[8 * c + 4] * f, o[8 * c + 5] * f, hi.z, lo.z);
        split2(o[8 * c + 6] * f, o[8 * c + 7] * f, hi.w, lo.w);
        const uint32_t at = core_off<HD>(lrow, half * (ND / 8) + c) / 16;
        sm.q[0][at] = hi;
        sm.q[1][at] = lo;
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] = 0.f;
    }
    // ---- the first tile
    convert(kc, sm.k);
    convert(vc, sm.v);
    if (tid < 8) put_scale(it & 1);
    tc::fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    if (uwarp == 0 && elect_one()) issue_s(it & 1);
    __syncwarp();
    load_codes(a.c.k, tile + 1, kc);
    load_codes(a.c.v, tile + 1, vc);
    load_scale(tile + 1);
    look(tile + 2);
    const bool warp_live = sm.seg.r * BM + 32 * (warp & 3) < sm.seg.cnt * a.group;

    for (; tile < stop; ++tile, ++it) {
      const bool more = tile + 1 < stop;
      const int base = tile * T;
      if (!lost && !tc::mbar_wait_sleep(mb_s, it & 1u)) lost = true;
      tc::fence_after_sync();
      const uint32_t cols = mine + T * (it & 1) + 32 * half;  // this thread's 32 scores: two blocks
      const bool edge = base + T - 1 > sm.seg.low || (a.window > 0 && base <= sm.seg.top - a.window);
      const int hi = lim - base - 32 * half, lo = a.window > 0 ? hi - a.window + 1 : 0;  // seen: lo <= column <= hi
      const float f[2] = {rs * sm.scales[it & 1][0][2 * half], rs * sm.scales[it & 1][0][2 * half + 1]};
      if (warp_live) {
        float tops[2];  // of the blocks
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float s[16], top = -INFINITY;
          tmem_ld16(cols + 16 * c, s);
          if (edge) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (16 * c + j <= hi && 16 * c + j >= lo) top = fmaxf(top, s[j] * f[c]);
          } else {
            float mc[2] = {fmaxf(s[0], s[1]), fmaxf(s[2], s[3])};
#pragma unroll
            for (int j = 4; j < 16; j += 4) {
              mc[0] = fmaxf(mc[0], fmaxf(s[j], s[j + 1]));
              mc[1] = fmaxf(mc[1], fmaxf(s[j + 2], s[j + 3]));
            }
            top = fmaxf(mc[0], mc[1]) * f[c];  // scales are not negative
          }
          tops[c] = top;
        }
        sm.ex[half][lrow] = make_float2(tops[0], tops[1]);
      }
      __syncthreads();  // the maximum of the row's other half
      float corr = 1.f;
      if (warp_live) {
        const float2 e0 = sm.ex[0][lrow], e1 = sm.ex[1][lrow];
        const float mn = fmaxf(m, fmaxf(fmaxf(e0.x, e0.y), fmaxf(e1.x, e1.y))), mu = mn == -INFINITY ? 0.f : mn;
        corr = ex2(m - mu);
        n += m - mu;
        m = mn;
        const float4 lgv = *reinterpret_cast<const float4*>(sm.scales[it & 1][2]);
        n = fmaxf(n, fmaxf(fmaxf((e0.x - mu) + lgv.x, (e0.y - mu) + lgv.y), fmaxf((e1.x - mu) + lgv.z, (e1.y - mu) + lgv.w)));
        float back, down;
        next_unit(n, ev, back, down);
        const bool huge = fabsf(mu) >= kHuge;
        const float bias = bias_of(mu, huge);
        float sum = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float vs = in_units(sm.scales[it & 1][1][2 * half + c], down);
          float s[16];
          tmem_ld16(cols + 16 * c, s);
          float fc = f[c];
          if (huge) {
#pragma unroll
            for (int j = 0; j < 16; ++j) s[j] *= fc;
            fc = 1.f;
          }
          uint32_t ph[8], pl[8];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float p0 = ex2(fmaf(s[j], fc, bias)), p1 = ex2(fmaf(s[j + 1], fc, bias));
            float y0 = p0 * vs, y1 = p1 * vs;
            if (edge) {  // whatever the scales
              const bool in0 = 16 * c + j <= hi && 16 * c + j >= lo, in1 = 16 * c + j + 1 <= hi && 16 * c + j + 1 >= lo;
              p0 = in0 ? p0 : 0.f;
              y0 = in0 ? y0 : 0.f;
              p1 = in1 ? p1 : 0.f;
              y1 = in1 ? y1 : 0.f;
            }
            sum += p0;
            sum1 += p1;
            split2(y0, y1, ph[j / 2], pl[j / 2]);
          }
          tmem_st8(cols + 16 * c, ph);
          tmem_st8(cols + 16 * c + 8, pl);
        }
        l = fmaf(l, corr, sum + sum1);
        corr *= back;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      tc::fence_before_sync();
      __syncthreads();
      if (uwarp == 0 && elect_one()) issue_o(it & 1);
      __syncwarp();
      if (more) {  // the next tile's scores
        convert(kc, sm.k);
        if (tid < 8) put_scale((it + 1) & 1);
        tell(tile + 2);
        tc::fence_proxy_async_smem();  // before the next loads, which it would wait for
        tc::fence_before_sync();
        __syncthreads();
        if (uwarp == 0 && elect_one()) issue_s((it + 1) & 1);
        __syncwarp();
      }
      if (more) {
        load_codes(a.c.k, tile + 2, kc);
        load_scale(tile + 2);
      }
      if (!lost && !tc::mbar_wait_sleep(mb_o, it & 1u)) lost = true;
      tc::fence_after_sync();
      if (more) {
        convert(vc, sm.v);
        tc::fence_proxy_async_smem();
        load_codes(a.c.v, tile + 2, vc);
        look(tile + 3);
      }
      if (warp_live) {
#pragma unroll
        for (int d0 = 0; d0 < ND; d0 += 16) {
          float t[16];
          tmem_ld16(mine + kColsO + ND * half + d0, t);
#pragma unroll
          for (int d = 0; d < 16; ++d) o[d0 + d] = fmaf(o[d0 + d], corr, t[d]);
        }
      }
      tc::fence_before_sync();
    }

    // ---- the end of this CTA's part of the walk
    const int t0 = sm.seg.t0, row = sm.seg.r * BM + lrow, rows = sm.seg.cnt * a.group;
    const bool whole = t0 == 0 && sm.seg.n == sm.seg.nt;
    const int64_t to = row < rows ? row_of(a, HD, (int64_t)a.n_heads * HD, sm.seg.row0, sm.seg.h, row) : 0;
    if (__syncthreads_or(lost)) l = NAN;  // every thread has read `ex`
    sm.ex[half][lrow].x = l;
    if (tid == 0) next_segment();
    __syncthreads();
    const float lt = l + sm.ex[half ^ 1][lrow].x;
    float* part = ma.parts + ((int64_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * part_floats(BM, HD);
    if (!whole && half == 0) {
      part[lrow] = m;
      part[BM + lrow] = lt;
    }
    if (!whole || row < rows) {
      const float unit = pow2(ev), f = whole ? inv_of(lt) * down_of(lt) : down_of(lt);
      float4* dst = reinterpret_cast<float4*>((whole ? a.out + to : part + 2 * BM + lrow * HD) + half * ND);
#pragma unroll
      for (int d = 0; d < ND; d += 4)
        dst[d / 4] = make_float4(o[d] * f * unit, o[d + 1] * f * unit, o[d + 2] * f * unit, o[d + 3] * f * unit);
    }
    __syncthreads();  // `ex` is read
  }
  tc::fence_before_sync();
  if (__syncthreads_or(lost) && tid == 0) {  // products that nobody waited for
    tc::mbar_wait(mb_s, (it - 1) & 1u);
    tc::mbar_wait(mb_o, (it - 1) & 1u);
  }
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kCols) : "memory");
}

// The parts of a cut walk of k_paged_many, in the CTAs' order: a warp to a row.
constexpr int kJoinRows = 8;  // warps of a block
template <int HD>
__global__ void __launch_bounds__(kJoinRows * 32) k_paged_join_many(ManyArgs ma) {
  constexpr int BM = kManyBm, kAtOnce = 8;
  using V = typename std::conditional<HD == 128, float4, float2>::type;
  pdl_wait();
  const AttnArgs& a = ma.a;
  const Cut* cut = ma.cuts + blockIdx.x;
  const int n = __ldcg(&cut->parts), lane = threadIdx.x & 31, r = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  if (n == 0) return;
  const int at = __ldcg(&cut->r) * BM + r;
  if (at >= __ldcg(&cut->cnt) * a.group) return;
  float m = -INFINITY, l = 0.f;
  float o[4] = {};
  for (int i0 = 0; i0 < n; i0 += kAtOnce) {
    float mc[kAtOnce], lc[kAtOnce];
    V oc[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float* p = ma.parts + ((int64_t)(blockIdx.x + i0 + i) * 2 + (i0 + i == 0 ? 1 : 0)) * part_floats(BM, HD);
      const bool live = i0 + i < n;
      mc[i] = live ? __ldcg(p + r) : -INFINITY;
      lc[i] = live ? __ldcg(p + BM + r) : 0.f;
      oc[i] = live ? __ldcg(reinterpret_cast<const V*>(p + 2 * BM + r * HD) + lane) : V{};
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, mc[i]);
    const float f = m == -INFINITY ? l : ex2(m - top), up = up_of(l);  // without a maximum l is 0 or NaN
    m = top;
    l *= f;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float g = mc[i] == -INFINITY ? lc[i] : ex2(mc[i] - top);
      l = fmaf(lc[i], g, l);
      mc[i] = g * up_of(lc[i]);
    }
    const float norm = down_of(l);
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] *= f * up * norm;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float* x = reinterpret_cast<const float*>(&oc[i]);
#pragma unroll
      for (int d = 0; d < (int)(sizeof(V) / 4); ++d) o[d] = fmaf(x[d], mc[i] * norm, o[d]);
    }
  }
  const float inv = inv_of(l);
  V out;
  float* x = reinterpret_cast<float*>(&out);
#pragma unroll
  for (int d = 0; d < (int)(sizeof(V) / 4); ++d) x[d] = o[d] * inv;
  reinterpret_cast<V*>(a.out + row_of(a, HD, (int64_t)a.n_heads * HD, __ldcg(&cut->row0), __ldcg(&cut->h), at))[lane] = out;
}

// ------------------------------------------------------------------ host
inline bool attn_shape_ok(const qd_paged_kv* kv, int n_heads, int n_tokens, int n_seqs) {
  return paged::cache_status(kv, n_seqs) == QD_OK && n_heads >= 1 && n_heads % kv->n_kv_heads == 0 &&
         n_heads / kv->n_kv_heads <= 16 && n_tokens >= 1 && n_tokens <= QD_MAX_GEMM_TOKENS;
}
// Blocks of 16 rows where sequences can have more than 8: against blocks of 8, 20 sequences of 3 x 4 rows, 8 heads of 128,
// 3000 positions 50 and 62 us, 8 of 8 x 4 rows of 6000 69 and 83; the other way round 4 of 8 x 3 rows, 3 heads of 64, 3000
// 13.6 and 12.2.  All sequences of a call have the same blocks, so that one of two tokens among 99 single ones of 32/8
// heads takes the call from 83 to 109 us.
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

// Whether a call takes the kernel for many rows: it can have sequences of so many (their rows are at most n_tokens
// x group, and a batch with no more tokens than sequences is taken to have one each), and there is work for it, counted
// in positions of a 16-row block as the cache has room for, a start as 1000 of them.  Few against many rows, in us:
//   1 head, 7 ragged sequences of 45 x 8 rows at most, 3000 positions (work 0.3e6)    14 33
//   8 heads, 20 x 4 rows, 20000 positions (0.8e6)                                     64 72
//   3 heads, 4 ragged sequences of 300 x 3 rows at most, 1500 positions (1.0e6)       31 41
//   8 heads, 64 x 4 rows, 32700 positions (4.3e6)                                    156 91
//   8 heads of 128, 1024 x 4 rows, 2040 positions (6.2e6)                            277 136
// These tables are as wide as the longest sequence.  The host knows neither the lengths nor what one sequence has of the
// rows, so that a wider table brings this kernel to shorter walks (20 tokens of one sequence at 1000, 32/8 heads of 128:
// 16 us with room for 2048 positions, 31 for 131072; 7 sequences of 45 rows at most, a window of 1000: 13 for 4032, 34 for
// 120000), and a batch without a sequence of so many rows pays for a list, a kernel and a join that find nothing (100
// of 4 tokens 100 and 110 us; 99 single tokens and one of two 109 and 119).
// The units of a head must fit an int.
constexpr int64_t kManyWork = 2000000;
inline bool has_many(int n_kv, int group, int n_tokens, int n_seqs, int capacity) {
  const int64_t rows = (int64_t)n_tokens * group;
  return rows > kFewRows && n_tokens > n_seqs && n_kv * ((rows + 15) / 16) * ((int64_t)capacity + 1000) > kManyWork &&
         (int64_t)most_blocks(group, n_tokens, n_seqs) * (capacity / kManyTile + 1 + kManyStart) < (1ll << 31);
}
inline int many_ctas() { return std::min(2 * attn_sm_count(), kMaxCtas); }

template <int HD, int FMT>
qd_status launch_many(const ManyArgs& m, cudaStream_t st) {
  using S = Many<HD>;
  static std::atomic<bool> done[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QD_ERR_CUDA;
  const auto kern = k_paged_many<HD, FMT>;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S)) != cudaSuccess)
      return QD_ERR_CUDA;
    done[dev] = true;
  }
  k_paged_list<<<1, kListThreads, 0, st>>>(m);
  kern<<<many_ctas(), kManyThreads, sizeof(S), st>>>(m);
  const qd_status s = launch_status();
  if (s != QD_OK) return s;
  return launch_k(k_paged_join_many<HD>, dim3((unsigned)many_ctas(), kManyBm / kJoinRows), dim3(kJoinRows * 32), 0, st, true, m);
}

template <int HD, int FMT>
qd_status launch_attn(AttnArgs a, cudaStream_t st) {
  if (has_many(a.c.n_kv, a.group, a.n_tokens, a.n_seqs, a.c.capacity)) {
    ManyArgs m;
    m.a = a;
    m.min_rows = a.n_seqs == 1 ? 1 : kFewRows + 1;
    m.most = most_blocks(a.group, a.n_tokens, a.n_seqs);
    m.ctas = many_ctas();
    unsigned char* at = reinterpret_cast<unsigned char*>(a.ws);  // one kernel's parts are joined before the other's begin
    m.cuts = reinterpret_cast<Cut*>(at);
    m.head = reinterpret_cast<ManyHead*>(at + kCutBytes);
    m.parts = reinterpret_cast<float*>(at + kCutBytes + align_up(list_bytes(a.group, a.n_tokens, a.n_seqs), 256));
    const qd_status s = launch_many<HD, FMT>(m, st);
    if (s != QD_OK || a.n_seqs == 1) return s;
    a.max_rows = kFewRows;
  }
  return rows16(a.group, a.n_tokens, a.n_seqs) ? launch_few<HD, FMT, true>(a, st) : launch_few<HD, FMT, false>(a, st);
}

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

size_t qd_paged_attn_workspace(const qd_paged_kv* kv, int n_heads, int n_tokens, int n_seqs) {
  if (!attn_shape_ok(kv, n_heads, n_tokens, n_seqs)) return 0;
  const int group = n_heads / kv->n_kv_heads;
  const size_t ctas = (size_t)std::min(attn_sm_count() * 3, kMaxCtas);  // of few rows, whatever the call
  const size_t few = ctas * 2 * part_floats(16, kv->head_dim) * sizeof(float);
  if ((int64_t)n_tokens * group <= kFewRows) return kCutBytes + few;
  const size_t many = align_up(list_bytes(group, n_tokens, n_seqs), 256) +
                      (size_t)many_ctas() * 2 * part_floats(kManyBm, kv->head_dim) * sizeof(float);
  return kCutBytes + std::max(few, many);
}

qd_status qd_paged_attn(const qd_paged_kv* kv, const float* q, int64_t q_stride, float* out, int n_heads, int n_tokens,
                        const int32_t* row_start, const int32_t* pos, int n_seqs, float scale, int window,
                        void* workspace, size_t workspace_bytes, qd_stream_t stream) {
  const float scale2 = scale * 1.4426950408889634f;  // scores in powers of two
  if (!q || !out || !row_start || !pos || !workspace || window < 0 || !std::isfinite(scale2)) return QD_ERR_INVALID_ARG;
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
  a.scale = scale2;
  a.window = window < a.c.capacity ? window : 0;  // a wider one hides nothing
  a.max_rows = 1 << 30;
  a.ws = static_cast<float*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  if (kv->head_dim == 64)
    return kv->fmt == QD_KV_I8 ? launch_attn<64, QD_KV_I8>(a, st) : launch_attn<64, QD_KV_E4M3>(a, st);
  return kv->fmt == QD_KV_I8 ? launch_attn<128, QD_KV_I8>(a, st) : launch_attn<128, QD_KV_E4M3>(a, st);
}

}  // extern "C"
