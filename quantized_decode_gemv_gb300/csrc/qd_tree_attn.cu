// Attention of a tree of drafted tokens over the cache: node i of sequence b sees the pos[b]
// cached positions and the draft slots j with bit j of its mask set,
//   o = sum_p softmax_p(q . k_p / sqrt(head_dim)) v_p.
//
// The rows that share a kv head (nodes x query heads of the group) walk its positions together
// with an online softmax: s = q k^T and o += p v are matrix products with f32 accumulators.
// Outputs are f32, and a binary16 operand alone is 2^-12 off, so what is f32 enters the products
// in parts, each the rounded rest of those before it.  A binary16 cache is exact as it is, and
//  - q has two binary16 parts, scaled by a power of two per row,
//  - the weights p = 2^(s - m + 15) too (the 2^15 cancels in o / l).
// A low part ends at binary16's subnormal step 2^-24, so a row's largest operand stands at 2^14 to
// 2^15: what is 2^-17 of it or more has 22 bits, and what is less is 2^-40 of it off.  (With q at 1
// to 2 and p at 2^12 at most those were 2^-3 and 2^-26 for q and 2^-14 and 2^-37 for p, in the same
// time; a dimension of q 2^14 times the others left them 12 bits.)
// That is 2 + 2 products a tile.  With an f32 cache all operands have two TF32 parts (2^-21, 3 + 3
// products, lo lo is dropped) or three bfloat16 ones (2^-26, 6 + 6), see each kernel: both types
// have f32's exponents, so what lies beside an element, and in the other rows, costs it nothing.
// Scores, running maxima, sums and o are f32.  The matrix units cut their f32 sums off instead of
// rounding them, so the low parts are summed first, a tile's products start from zero, and they
// are added to o with rounded f32 additions (one accumulator through a walk of 4080 positions:
// 1.4e-6 relative error of o instead of 4e-7).
//
// Work: the walks of all (sequence, kv head, block of rows) are laid end to end in units of a
// tile and cut evenly over the CTAs, whatever the lengths; a walk's start (its queries, its
// result) counts as kStart units.  A CTA that holds a part of a walk writes (m, l, o) to the
// workspace and a second kernel joins the parts in order.  Where the cache has room for at most
// kWholeTiles tiles a walk, no walk is cut and there is one launch.
//
// What bounds it: HBM for few rows on long caches, for many rows the latency of a tile's dependent
// steps (1.8 of 4 instructions a cycle, the tensor pipe active 32 to 40 %), launch and a few tiles'
// latency for short caches.  Measured on one GB300 (floor: the bytes at 6.77 TB/s or the products at
// 1946 TFLOP/s, counted once):
//   9/3 heads, 8 nodes, 100 positions, f32              8.2 us (floor 0.03)
//   32/32 heads, 16 nodes, 4080 positions, f32           21 us (10.0)
//   the same, 16 sequences of 4095, f32                 195 us (160)
//   the same, 16 ragged sequences, binary16              53 us (40)
//   32/8 heads, 64 nodes, 32700 positions, binary16      59 us (10)
//   64/8 heads, 64 nodes, 8000 positions, f32            68 us (4.9)
//   8/1 heads, 27 nodes, 5 ragged sequences, f32         18 us (0.6)
// The unit counts, in us: kStart 3 against 5 at 4080 positions 20.6 and 22.6, against 2 20.6 and 21.2, at
// 32/32 heads, 64 nodes and 1000 positions f32 25.1 and 22.3, at 3/1 heads, 5 nodes and 4000 positions
// binary16 7.9 and 8.9.  kMinPer 2 against 1 at 3/1 heads, 5 nodes and 16000 positions f32
// 12.1 and 13.9, 1000 positions 9.4 and 8.4.  kWholeTiles 4 against 2 at 32 heads, 64 nodes and 100
// positions of 260 f32 9.5 and 13.7, 200 positions 11.0 and 15.0; one head, 300 of 364 12.1 and 8.7;
// against 8 at 9/3 heads and 370 positions 10.3 and 13.6.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "qd_internal.cuh"
#include "qd_tc.cuh"

namespace qd {
namespace {

constexpr int kHd = 64;
constexpr int kTile = 64;      // positions of the smallest tile of a whole CTA; the drafts are one tile
constexpr int kThreads = 128;  // of the join
constexpr float kBias = 15.f;  // log2 of the weights' scale on a binary16 cache
constexpr int kMinPer = 2;     // units of a CTA at least
constexpr int kWholeTiles = 4;  // walks of at most so many tiles are not cut
constexpr int kStart = 3;      // what the start of a walk costs, in tiles

// k_tree_attn_16: warps with tiles of their own, 6 of 16 positions (f32 cache) or 4 of 32; what
// they do side by side is one unit of work
__host__ __device__ constexpr int sub_positions(bool f16) { return f16 ? 32 : 16; }
__host__ __device__ constexpr int sub_warps(int sub) { return sub == 32 ? 4 : 6; }
static_assert(QD_MAX_TREE <= kTile, "the drafts fit one tile");

struct TreeAttnArgs {
  const float* q;
  int64_t q_batch_stride;
  const void *kc, *vc, *kd, *vd;
  float* out;
  int n_kv, group;
  const int32_t* pos;
  const uint64_t* mask;
  const int32_t* n_valid;
  int n_nodes, max_ctx, batch;
  float* ws;
  int blocks;  // of rows, at most
  int whole;   // 1: a CTA takes one whole walk
};

// Work of the sequences: nt tiles for each of n_kv * rb walks (0 when pos is out of range).
struct Plan {
  int off[QD_MAX_BATCH + 1];  // in units
  int nt[QD_MAX_BATCH], rb[QD_MAX_BATCH], p0[QD_MAX_BATCH], cnt[QD_MAX_BATCH];
};

// Tiles of a walk over p0 cached positions and cnt drafts; sub: sub_positions, or minus the
// positions of a tile that the whole CTA takes (the drafts are one such tile).
__host__ __device__ constexpr int walk_tiles(int sub, int p0, int cnt) {
  return sub > 0 ? ((p0 + sub - 1) / sub + (cnt + sub - 1) / sub + sub_warps(sub) - 1) / sub_warps(sub)
                 : (p0 - sub - 1) / -sub + 1;
}
// Filled by one warp; `bm` rows to a block.
template <int SUB>
__device__ __forceinline__ void make_plan(const TreeAttnArgs& a, int bm, Plan* p) {
  const int b = threadIdx.x & 31;
  int units = 0;
  if (b < a.batch) {
    const int cnt = a.n_valid ? min(max(a.n_valid[b], 0), a.n_nodes) : a.n_nodes;
    const int p0 = a.pos[b];
    const int rb = (cnt * a.group + bm - 1) / bm;
    const int nt = p0 < 0 || p0 > a.max_ctx ? 0 : walk_tiles(SUB, p0, cnt);
    p->cnt[b] = cnt;
    p->p0[b] = p0;
    p->rb[b] = rb;
    p->nt[b] = nt;
    units = nt ? (nt + kStart) * rb * a.n_kv : 0;
  }
  int sum = units;
#pragma unroll
  for (int o = 1; o < QD_MAX_BATCH; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (b >= o) sum += v;
  }
  if (b < QD_MAX_BATCH) p->off[b + 1] = sum;
  if (b == 0) p->off[0] = 0;
}
__device__ __forceinline__ int units_per_cta(int total, int ctas) { return max((total + ctas - 1) / ctas, kMinPer); }

// Row `at` (node, head of the group) of a walk, in q or out of sequence c.b.
template <typename C>
__device__ __forceinline__ float* row_of(const TreeAttnArgs& a, float* out, const C& c, int at) {
  const int node = at / a.group, g = at % a.group;
  return out + (((int64_t)c.b * a.n_nodes + node) * a.n_kv * a.group + c.h * a.group + g) * kHd;
}

// Floats of one partial: m and l of each row, then o.
__host__ __device__ constexpr int part_floats(int bm) { return bm * (kHd + 2); }

// ------------------------------------------------------------------ building blocks
// 16 bytes global -> shared, or 16 zero bytes
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
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
// Exponent e of a largest magnitude (given by its bits), so that x 2^-e is in 2^14 .. 2^15 (less for
// one under 2^-100); an infinity or NaN stays what it is.
__device__ __forceinline__ int scale_exp(uint32_t abs_bits) {
  return min(max((int)(abs_bits >> 23) - 127, -100), 127) - 14;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;
__device__ __forceinline__ uint32_t abs_max(float4 x) {
  return max(max(abs_bits(x.x), abs_bits(x.y)), max(abs_bits(x.z), abs_bits(x.w)));
}

// Byte offset of 16-byte chunk c of row r in a tile of 64 rows of 64 binary16 values: chunks
// permuted within a row so that 8 rows' same chunk (a matrix of ldmatrix) hits all banks.
__device__ __forceinline__ uint32_t tile_off(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// A CTA's place in the units: the tile t of a walk (sequence, kv head, block of rows) and its
// unit; with it the walk's tiles, positions and drafts, and the number of its kv head.
struct Cursor {
  int b, h, r, t, u;
  int nt, p0, cnt;
  int64_t head;
  __device__ __forceinline__ void enter(const Plan& p, int n_kv) {
    nt = p.nt[b];
    p0 = p.p0[b];
    cnt = p.cnt[b];
    head = (int64_t)b * n_kv + h;
  }
};
// The first tile at or behind unit u.
__device__ __forceinline__ Cursor cursor_at(const Plan& p, int n_kv, int u) {
  Cursor c;
  c.b = 0;
  while (u >= p.off[c.b + 1]) ++c.b;  // u < off[QD_MAX_BATCH]
  const int len = p.nt[c.b] + kStart, in = u - p.off[c.b], walk = in / len;
  c.t = max(in % len - kStart, 0);
  c.u = p.off[c.b] + walk * len + kStart + c.t;
  c.h = walk / p.rb[c.b];
  c.r = walk % p.rb[c.b];
  c.enter(p, n_kv);
  return c;
}
__device__ __forceinline__ void advance(const Plan& p, int n_kv, Cursor& c) {
  ++c.u;
  if (++c.t < c.nt) return;
  c.u += kStart;
  c.t = 0;
  if (++c.r < p.rb[c.b]) return;
  c.r = 0;
  if (++c.h == n_kv) {
    c.h = 0;
    do ++c.b;
    while (c.b < QD_MAX_BATCH - 1 && p.off[c.b] == p.off[c.b + 1]);
    if (c.b == QD_MAX_BATCH) return;  // behind the last one
  }
  c.enter(p, n_kv);
}

// This CTA's first tile and the unit at which it ends; false if it has none (and zeros written
// for a whole walk whose position is out of range).
template <int BM>
__device__ __forceinline__ bool first_tile(const TreeAttnArgs& a, const Plan& p, Cursor& cur, int& end) {
  if (!a.whole) {
    const int total = p.off[QD_MAX_BATCH];
    const int per = units_per_cta(total, gridDim.x);
    const int64_t first = (int64_t)blockIdx.x * per;
    if (first >= total) return false;
    end = min((int)first + per, total);
    cur = cursor_at(p, a.n_kv, (int)first);
    return cur.u < end;
  }
  const int walk = blockIdx.x;
  cur.b = walk / (a.n_kv * a.blocks);
  cur.h = walk / a.blocks % a.n_kv;
  cur.r = walk % a.blocks;
  cur.t = cur.u = 0;
  if (cur.r >= p.rb[cur.b]) return false;
  cur.enter(p, a.n_kv);
  end = cur.nt;
  if (end) return true;
  const int rows = cur.cnt * a.group;
  for (int x = threadIdx.x; x < BM * (kHd / 4); x += blockDim.x) {
    const int at = cur.r * BM + x / (kHd / 4);
    if (at < rows)
      reinterpret_cast<float4*>(row_of(a, a.out, cur, at))[x % (kHd / 4)] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  return false;
}

// ------------------------------------------------------------------ 16 rows
// Few rows to a kv head, or little work: blocks of 16, and warps that walk the positions side by side, each with
// tiles and a ring of its own (no barrier until the walk's end, where the warps' results are
// joined while the next walk's queries arrive).  A binary16 cache as above, 4 warps with 32
// positions a tile.  An f32 cache without a conversion in shared memory, 6 warps with 16
// positions: m16n8k8 TF32 products, each f32 operand as two TF32 parts (hi = the upper 10
// fraction bits, lo = as many of the rest: 2^-21 off), hi hi + lo hi + hi lo.  TF32 keeps
// f32's exponents, so nothing is scaled; the products run at half the binary16 rate, which 16
// rows leave room for.  What bounds it is a warp's chain of dependent instructions (about 700 a
// tile), hidden by the other warps, and the start and end of a walk, hidden by the SM's other CTA:
// two CTAs of 4 warps against one of 8, 62 -> 54 us for 16 ragged sequences; two of 6 with the
// queries' fragments in shared memory against one of 8 with them in registers, 203 -> 183 us for
// 16 x 32 heads of 4095 positions f32 (before lo was rounded); 12 warps spill on a binary16 cache.
// A conversion pass through shared memory and binary16 parts instead of TF32: 33 against 23 us for
// one sequence.
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// The product reads the upper 10 fraction bits of its operands and cuts the rest off.  For the
// scores hi is rounded, so that lo is half as large; for the values lo is, which is a shorter
// chain.  Cutting both off left k and q 7e-8 too small on average, which a score of 10 makes 1e-6
// of its weight.  Error of o against 64 bits over the plain f32 form's, and the time for 16 x 32
// heads of 4095 positions: as here 0.9 and 193 us, hi rounded everywhere 0.9 and 205 us, lo
// rounded everywhere 1.2 and 194 us, both cut off 2.0 and 183 us.
template <bool SCORES = false>
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + (SCORES ? 0x1000u : 0u)) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + (SCORES ? 0u : 0x1000u);  // one of the two is NaN where x is
}
// f32 rows of 256 bytes: 16-byte chunk c of row r stands at c ^ swz(r), so that both reads hit
// all banks: k (8 rows at one chunk of each lane's four) and v (every second row at two chunks).
__device__ __forceinline__ int swz(int r) { return ((r >> 1) & 1) | ((((r >> 2) ^ r) & 1) << 2); }

template <bool F16>
struct Smem16 {
  static constexpr int kWarps = sub_warps(sub_positions(F16)), kStages = F16 ? 3 : 2;
  static constexpr int kRowBytes = F16 ? 128 : 256;
  uint4 ring[kWarps][kStages][2][sub_positions(F16) * kRowBytes / 16];  // K, V; m, l, o of a share at a walk's end
  uint4 q[F16 ? 4 : 8][2][32];  // the fragments of q's k steps, hi and lo, by lane
  Plan plan;
};

template <bool F16>
__global__ void __launch_bounds__(Smem16<F16>::kWarps * 32, 2) k_tree_attn_16(TreeAttnArgs a) {
  using KV = typename std::conditional<F16, __half, float>::type;
  using S = Smem16<F16>;
  constexpr int kSub = sub_positions(F16), NT = kSub / 8, kWarps16 = S::kWarps;
  constexpr int kRow = S::kRowBytes;
  constexpr int kLag = S::kStages - 1;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qr = lane >> 2, qc = lane & 3;

  pdl_trigger();
  if (warp == 0) make_plan<kSub>(a, 16, &sm.plan);
  __syncthreads();
  Cursor cur;
  int end;
  if (!first_tile<16>(a, sm.plan, cur, end)) return;
  Cursor pre = cur;

  const KV* kc = static_cast<const KV*>(a.kc);
  const KV* vc = static_cast<const KV*>(a.vc);
  const KV* kd = static_cast<const KV*>(a.kd);
  const KV* vd = static_cast<const KV*>(a.vd);

  // this warp's positions of the unit at `pre` into ring slot s (zeros behind their end), and
  // on to the next unit
  auto produce = [&](int s) {
    if (pre.u < end) {
      const int p0 = pre.p0, cnt = pre.cnt;
      const int np = (p0 + kSub - 1) / kSub, sub = pre.t * kWarps16 + warp;
      const bool draft = sub >= np;
      const int row0 = (draft ? sub - np : sub) * kSub;
      const int rows = (draft ? cnt : p0) - row0;
      if (rows > 0) {
        const int64_t base = (pre.head * (draft ? a.n_nodes : a.max_ctx) + row0) * kHd;
        const KV* ks = (draft ? kd : kc) + base;
        const KV* vs = (draft ? vd : vc) + base;
        const uint32_t dk = tc::smem_u32(sm.ring[warp][s][0]), dv = tc::smem_u32(sm.ring[warp][s][1]);
        constexpr int kPer = kRow / 16;
        const int c = lane % kPer, r0 = lane / kPer;
        const int first = r0 * kHd + c * (16 / (int)sizeof(KV));
#pragma unroll
        for (int i = 0; i < kSub * kPer / 32; ++i) {
          const int r = r0 + i * (32 / kPer);
          const uint32_t off = F16 ? tile_off(r, c) : (uint32_t)(r * kRow + ((c ^ swz(r)) << 4));
          if (rows >= kSub) {
            cp16(dk + off, ks + first + i * (32 / kPer) * kHd);
            cp16(dv + off, vs + first + i * (32 / kPer) * kHd);
          } else {
            const bool live = r < rows;
            const int src = live ? r * kHd + c * (16 / (int)sizeof(KV)) : 0;
            cp16(dk + off, ks + src, live);
            cp16(dv + off, vs + src, live);
          }
        }
      }
      advance(sm.plan, a.n_kv, pre);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kLag; ++s) produce(s);

  float o[8][4];
  float m[2], l[2], rs[2] = {1.f, 1.f};
  uint64_t vis[2];
  int t_begin = -1;

  // a walk's queries and masks: asked for ...
  float4 x[2][4];
  auto load_q = [&](const Cursor& c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = c.r * 16 + qr + 8 * i, node = at / a.group, g = at % a.group;
      const bool live = at < c.cnt * a.group;
      const float4* src = reinterpret_cast<const float4*>(
          a.q + (int64_t)c.b * a.q_batch_stride + ((int64_t)node * a.n_kv * a.group + c.h * a.group + g) * kHd);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = live ? __ldcg(src + qc + 4 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
      vis[i] = live ? a.mask[(int64_t)c.b * a.n_nodes + node] : 0ull;
      if (c.cnt < 64) vis[i] &= (1ull << c.cnt) - 1;
    }
  };
  // ... and made operands in shared memory by warp 0 (in registers they leave no room for 12
  // warps).  The lane has dims 4 (qc + 4 j) .. + 3 of its rows; f32 cache: k step 2 j + e / 2 has
  // them at k = qc and qc + 4.
  auto set_q = [&]() {
    const float scale = 1.4426950408889634f * 0.125f;  // scores in log2 units
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (F16) {
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j].x *= scale;
          x[i][j].y *= scale;
          x[i][j].z *= scale;
          x[i][j].w *= scale;
          mx = max(mx, abs_max(x[i][j]));
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = scale_exp(mx);
        rs[i] = pow2(e);
        const float f = pow2(-e);
        if (warp == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // dims 16 j + 4 qc .. + 3 as pairs 2 qc, 2 qc + 1 of k step j; pair p belongs to lane p & 3
            uint32_t hi, lo;
            uint32_t* to0 = reinterpret_cast<uint32_t*>(&sm.q[j][0][(lane & 28) | (2 * qc & 3)]);
            uint32_t* to1 = reinterpret_cast<uint32_t*>(&sm.q[j][1][(lane & 28) | (2 * qc & 3)]);
            const int at = i + 2 * (qc >> 1);
            split2(x[i][j].x * f, x[i][j].y * f, hi, lo);
            to0[at] = hi;
            to1[at] = lo;
            split2(x[i][j].z * f, x[i][j].w * f, hi, lo);
            to0[4 + at] = hi;
            to1[4 + at] = lo;
          }
        }
      } else {
        if (warp == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            auto in = [scale](float f) { return (f + (f - f)) * scale; };  // an infinity is a NaN too
            auto put = [&](int ks, int e, float f) {
              uint32_t hi, lo;
              split_tf32<true>(in(f), hi, lo);
              reinterpret_cast<uint32_t*>(&sm.q[ks][0][lane])[e] = hi;
              reinterpret_cast<uint32_t*>(&sm.q[ks][1][lane])[e] = lo;
            };
            put(2 * j, i, x[i][j].x);
            put(2 * j, i + 2, x[i][j].y);
            put(2 * j + 1, i, x[i][j].z);
            put(2 * j + 1, i + 2, x[i][j].w);
          }
        }
      }
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
  };
  load_q(cur);
  set_q();
  __syncthreads();

  for (int it = 0; cur.u < end; ++it) {
    const int p0 = cur.p0, cnt = cur.cnt, nt = cur.nt;
    const bool last = cur.t == nt - 1;
    const bool more = cur.u + 1 + (last ? kStart : 0) < end;
    if (t_begin < 0) t_begin = cur.t;

    // ---- this warp's positions
    const int slot = it % S::kStages;
    cp_wait<kLag - 1>();
    __syncwarp();  // every lane's copies have landed, and the slot before this one has been read
    produce((it + kLag) % S::kStages);
    const int np = (p0 + kSub - 1) / kSub, sub = cur.t * kWarps16 + warp;
    const bool draft = sub >= np;
    const int row0 = (draft ? sub - np : sub) * kSub;
    const int left = (draft ? cnt : p0) - row0;
    if (left > 0) {
      const uint32_t kt = tc::smem_u32(sm.ring[warp][slot][0]), vt = tc::smem_u32(sm.ring[warp][slot][1]);
      const unsigned char* kp = reinterpret_cast<const unsigned char*>(sm.ring[warp][slot][0]);
      const unsigned char* vp = reinterpret_cast<const unsigned char*>(sm.ring[warp][slot][1]);
      float s[NT][4], sl[NT][4];
      if constexpr (F16) {
        const int kr = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint4 vh = sm.q[ks][0][lane], vl = sm.q[ks][1][lane];
          const uint32_t fh[4] = {vh.x, vh.y, vh.z, vh.w}, fl[4] = {vl.x, vl.y, vl.z, vl.w};
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm4(kt + tile_off(kr + 8 * n, 2 * ks + ((lane >> 3) & 1)), b);
            if (ks == 0) {
              mma0(s[n], fh, b[0], b[1]);
              mma0(s[n + 1], fh, b[2], b[3]);
              mma0(sl[n], fl, b[0], b[1]);
              mma0(sl[n + 1], fl, b[2], b[3]);
            } else {
              mma(s[n], fh, b[0], b[1]);
              mma(s[n + 1], fh, b[2], b[3]);
              mma(sl[n], fl, b[0], b[1]);
              mma(sl[n + 1], fl, b[2], b[3]);
            }
          }
        }
      } else {
        float sx[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t bh[2][4], bl[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int r = 8 * n + qr;
            const float4 x = *reinterpret_cast<const float4*>(kp + r * kRow + (((qc + 4 * j) ^ swz(r)) << 4));
            split_tf32<true>(x.x, bh[n][0], bl[n][0]);
            split_tf32<true>(x.y, bh[n][1], bl[n][1]);
            split_tf32<true>(x.z, bh[n][2], bl[n][2]);
            split_tf32<true>(x.w, bh[n][3], bl[n][3]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 vh = sm.q[2 * j + h][0][lane], vl = sm.q[2 * j + h][1][lane];
            const uint32_t fh[4] = {vh.x, vh.y, vh.z, vh.w}, fl[4] = {vl.x, vl.y, vl.z, vl.w};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              if (j == 0 && h == 0) {
                mma8_0(s[n], fh, bh[n][0], bh[n][1]);
                mma8_0(sl[n], fl, bh[n][0], bh[n][1]);
                mma8_0(sx[n], fh, bl[n][0], bl[n][1]);
              } else {
                mma8(s[n], fh, bh[n][2 * h], bh[n][2 * h + 1]);
                mma8(sl[n], fl, bh[n][2 * h], bh[n][2 * h + 1]);
                mma8(sx[n], fh, bl[n][2 * h], bl[n][2 * h + 1]);
              }
            }
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sl[n][e] += sx[n][e];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] += sl[n][e];
      if (draft || left < kSub) {
        const uint32_t in = left < kSub ? (1u << left) - 1 : ~0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t see = (draft ? (uint32_t)(vis[i] >> row0) : in) >> (2 * qc);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (!(see >> (8 * n) & 1)) s[n][2 * i] = -INFINITY;
            if (!(see >> (8 * n + 1) & 1)) s[n][2 * i + 1] = -INFINITY;
          }
        }
      }
      float corr[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
        for (int n = 1; n < NT; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[i], mx * rs[i]);
        const float mu = mn == -INFINITY ? 0.f : mn;
        corr[i] = ex2(m[i] - mu);
        m[i] = mn;
        const float bias = (F16 ? kBias : 0.f) - mu;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[n][2 * i + e] = ex2(fmaf(s[n][2 * i + e], rs[i], bias));
            sum += s[n][2 * i + e];
          }
        l[i] = fmaf(l[i], corr[i], sum);
      }

      // draft rows whose values hold an infinity or NaN are taken out of the product and added
      // where they are seen
      uint32_t bad = 0;
      if (draft) {
        bool off = false;  // half a row of f32 or a row of binary16 to a lane
        uint4* row = reinterpret_cast<uint4*>(sm.ring[warp][slot][1]) + lane * 8;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 w = row[c];
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            off |= F16 ? ((u[e] & 0x7C00u) == 0x7C00u || (u[e] & 0x7C000000u) == 0x7C000000u)
                       : (u[e] & kInfBits) == kInfBits;
        }
        const uint32_t any = __ballot_sync(0xffffffffu, off);
        if (any) {
          bad = any;
          if (!F16) {
            bad = 0;
#pragma unroll
            for (int r = 0; r < kSub; ++r) bad |= (any >> (2 * r & 31) & 3u ? 1u : 0u) << r;
          }
          if (bad >> (F16 ? lane : lane >> 1) & 1) {
#pragma unroll
            for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
          const KV* vrow = vd + (((int64_t)cur.b * a.n_kv + cur.h) * a.n_nodes + row0) * kHd;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if ((vis[i] >> row0) & bad) {  // the other rows keep every bit
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[d][2 * i] *= corr[i];
                o[d][2 * i + 1] *= corr[i];
              }
              corr[i] = 1.f;
            }
#pragma unroll
          for (int r = 0; r < kSub; ++r) {
            if (!(bad >> r & 1)) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p = __shfl_sync(0xffffffffu, s[r / 8][2 * i + (r & 1)], (lane & 28) | ((r & 7) >> 1));
              if (!(vis[i] >> (row0 + r) & 1)) continue;
#pragma unroll
              for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  o[d][2 * i + e] += p * (float)vrow[r * kHd + (F16 ? 8 * d + 2 * qc + e : 16 * qc + 8 * e + d)];
            }
          }
        }
      }

      if constexpr (F16) {
        uint32_t ph[NT / 2][4], pl[NT / 2][4];
#pragma unroll
        for (int k = 0; k < NT / 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            split2(s[2 * k + (e >> 1)][2 * (e & 1)], s[2 * k + (e >> 1)][2 * (e & 1) + 1], ph[k][e], pl[k][e]);
        const int vr = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int d = 0; d < 8; d += 4) {
          uint32_t b[NT / 2][2][4];
          float t[4][4];
#pragma unroll
          for (int k = 0; k < NT / 2; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) ldsm4t(vt + tile_off(vr + 16 * k, d + 2 * x + ((lane >> 4) & 1)), b[k][x]);
          // the low parts first: what is cut off there does not count
#pragma unroll
          for (int k = 0; k < NT / 2; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (k == 0)
                mma0(t[x], pl[k], b[k][x >> 1][2 * (x & 1)], b[k][x >> 1][2 * (x & 1) + 1]);
              else
                mma(t[x], pl[k], b[k][x >> 1][2 * (x & 1)], b[k][x >> 1][2 * (x & 1) + 1]);
#pragma unroll
          for (int k = 0; k < NT / 2; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) mma(t[x], ph[k], b[k][x >> 1][2 * (x & 1)], b[k][x >> 1][2 * (x & 1) + 1]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d + x][e] = fmaf(o[d + x][e], corr[e >> 1], t[x][e]);
        }
      } else {
        // k = qc of step t is position 8 t + 2 qc, k = qc + 4 the one after it; column n of
        // product d is dim 8 n + d, so a lane's values are two chunks of each row
        uint32_t ph[2][4], pl[2][4];
        float v[2][2][8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          split_tf32(s[t][0], ph[t][0], pl[t][0]);
          split_tf32(s[t][2], ph[t][1], pl[t][1]);
          split_tf32(s[t][1], ph[t][2], pl[t][2]);
          split_tf32(s[t][3], ph[t][3], pl[t][3]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * t + 2 * qc + e;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float4 x = *reinterpret_cast<const float4*>(vp + r * kRow + (((2 * qr + c) ^ swz(r)) << 4));
              v[t][e][4 * c] = x.x;
              v[t][e][4 * c + 1] = x.y;
              v[t][e][4 * c + 2] = x.z;
              v[t][e][4 * c + 3] = x.w;
            }
          }
        }
        // four products at a time, so that one's chain runs in the shadow of the others'
#pragma unroll
        for (int d0 = 0; d0 < 8; d0 += 4) {
          uint32_t h[4][2][2], w[4][2][2];
          float t0[4][4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) split_tf32(v[t][e][d0 + x], h[x][t][e], w[x][t][e]);
          // the low parts first: what is cut off there does not count
#pragma unroll
          for (int x = 0; x < 4; ++x) mma8_0(t0[x], pl[0], h[x][0][0], h[x][0][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) mma8(t0[x], pl[1], h[x][1][0], h[x][1][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) mma8(t0[x], ph[0], w[x][0][0], w[x][0][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) mma8(t0[x], ph[1], w[x][1][0], w[x][1][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) mma8(t0[x], ph[0], h[x][0][0], h[x][0][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) mma8(t0[x], ph[1], h[x][1][0], h[x][1][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d0 + x][e] = fmaf(o[d0 + x][e], corr[e >> 1], t0[x][e]);
        }
      }
    }

    // ---- the end of this CTA's part of the walk
    if (last || !more) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      }
      const Cursor done = cur;
      const bool whole = t_begin == 0 && last;
      const int part_slot = t_begin > 0 ? 0 : 1;
      // the share goes to this warp's ring slot, which it has read and the next tile but one will
      // fill; pair c of a row at c ^ 4 (row & 7): no bank twice
      auto share = [&](int w) { return reinterpret_cast<float*>(sm.ring[w][slot][0]); };
      static_assert(sizeof(sm.ring[0][0]) >= part_floats(16) * 4, "a share fits a slot");
      __syncwarp();
      {
        float* mine = share(warp);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = qr + 8 * i;
          if (qc == 0) {
            mine[r] = m[i];
            mine[16 + r] = l[i];
          }
          float2* dst = reinterpret_cast<float2*>(mine + 32 + r * kHd);
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            if constexpr (F16)
              dst[(4 * d + qc) ^ (4 * qr)] = make_float2(o[d][2 * i], o[d][2 * i + 1]);
            else  // dims 16 qc + 8 e + 2 k, + 1
              dst[(8 * qc + d) ^ (4 * qr)] =
                  make_float2(o[2 * (d & 3)][2 * i + (d >> 2)], o[2 * (d & 3) + 1][2 * i + (d >> 2)]);
          }
        }
      }
      advance(sm.plan, a.n_kv, cur);
      if (more) load_q(cur);  // on its way meanwhile
      __syncthreads();
      const int done_rows = done.cnt * a.group;
      for (int r = warp; r < 16; r += kWarps16) {
        float mt = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps16; ++w) mt = fmaxf(mt, share(w)[r]);
        float lt = 0.f;
        float2 ot = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps16; ++w) {
          const float mw = share(w)[r], lw = share(w)[16 + r];
          const float f = mw == -INFINITY ? lw : ex2(mw - mt);  // a share without a maximum has l = 0 or NaN
          const float2 ow = reinterpret_cast<const float2*>(share(w) + 32 + r * kHd)[lane ^ (4 * (r & 7))];
          lt = fmaf(lw, f, lt);
          ot.x = fmaf(ow.x, f, ot.x);
          ot.y = fmaf(ow.y, f, ot.y);
        }
        if (whole) {
          if (done.r * 16 + r < done_rows) {
            const float inv = 1.f / lt;
            reinterpret_cast<float2*>(row_of(a, a.out, done, done.r * 16 + r))[lane] =
                lt == 0.f ? make_float2(0.f, 0.f) : make_float2(ot.x * inv, ot.y * inv);
          }
        } else {
          float* part = a.ws + ((int64_t)blockIdx.x * 2 + part_slot) * part_floats(16);
          if (lane == 0) {
            part[r] = mt;
            part[16 + r] = lt;
          }
          reinterpret_cast<float2*>(part + 32 + r * kHd)[lane] = ot;
        }
      }
      if (more) set_q();
      __syncthreads();  // every share has been read, and q stands
      t_begin = -1;
    } else {
      advance(sm.plan, a.n_kv, cur);
    }
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------ 128 rows
// Many rows to a kv head and much work: blocks of 128 on the 5th-generation tensor cores, two threads to a row.
// Per tile (128 positions of a binary16 cache, 64 of an f32 one) one thread issues s = q k^T
// (tcgen05.mma, M = 128, q in tensor memory, K in shared memory) into tensor memory; a row's
// threads read half of its scores each (tcgen05.ld), exchange their maxima, read the scores again
// 16 at a time (the registers have to do for two CTAs to an SM, and the shared memory leaves
// spills no L1; 36 bytes of the binary16 kernel's still spill) and write the weights' parts over
// them as the A operand of o = p v, a third one beside them (V as it lies, [position][dim], is the
// transposed B operand); each adds 32 dims of the tile's o to its own registers, rounded.
// Two CTAs to an SM, one's products under the other's softmax.
// A binary16 tile lies in the TMA's 128-byte swizzle; an f32 one is converted into 8 x 8 core
// matrices of 128 bytes: row r, 16-byte chunk c at core_off(r, c).
// Operands beside an f32 cache: hi, mid and lo of bfloat16, rounded, so that the products that are
// left out (mid lo, lo mid, lo lo) are 2^-26 of the whole and of either sign.  68.1 us for 8 x 512
// rows of 8000 positions; two binary16 parts with a power of two for each position, half as many
// products but maxima and scales to find, took 69.6 us, an element far below its row's largest lost
// digits, and so did all values beside a row of 10^5 times their size, whatever its weight.
constexpr int kThreads128 = 256;
__device__ __forceinline__ uint32_t core_off(int r, int c) {
  return (uint32_t)((((r >> 3) * 8 + c) * 128) + (r & 7) * 16);
}
__host__ __device__ constexpr int tile128(bool f16) { return f16 ? 128 : 64; }
constexpr uint32_t kIdescBf16 = (1u << 7) | (1u << 10);              // A and B of bfloat16
constexpr uint32_t kIdescO = tc::idesc_f16(128, kHd) | (1u << 16);  // B with N contiguous
constexpr uint32_t kFarBits = 0x7F000000u;                           // 2^127: a bfloat16 part may be an infinity
// The next bfloat16 part of (x, y), taken off them.
__device__ __forceinline__ uint32_t bf16_part(float2& x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
  x.x -= __uint_as_float(u << 16);
  x.y -= __uint_as_float(u & 0xFFFF0000u);
  return u;
}
// One lane of the (whole) calling warp.
__device__ __forceinline__ bool elect_one() {
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

// two f32 operations at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n"
      ".reg .b64 a, b, c, d;\n"
      "mov.b64 a, {%2, %3};\n"
      "mov.b64 b, {%4, %5};\n"
      "mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\n"
      "mov.b64 {%0, %1}, d;\n"
      "}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n"
      ".reg .b64 a, b, d;\n"
      "mov.b64 a, {%2, %3};\n"
      "mov.b64 b, {%4, %5};\n"
      "add.rn.f32x2 d, a, b;\n"
      "mov.b64 {%0, %1}, d;\n"
      "}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// What a CTA does with a tile.  One thread steps through the units and leaves it here a tile
// ahead; with a cursor in every thread's registers the kernel spilled, and the shared memory
// leaves spills no L1 to stay in.
struct Tile128 {
  int64_t base;           // its rows in the caches (drafts: in the draft buffers), in elements
  int rows, left;         // rows that exist; cached positions from its first one on
  int b, h, r, cnt;
  int draft, begin, last, whole, slot, valid;  // begin / last of this CTA's part of the walk; slot of the part
};

// K and V of a binary16 cache, and of the draft buffers, as rows of 64 values (128 bytes) that a
// TMA load leaves in the 128-byte swizzle: chunk c of row r at c ^ (r & 7).
struct Maps128 {
  CUtensorMap m[4];  // k cache, v cache, k draft, v draft
};
constexpr int kBoxRows = 64;
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int row, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(row), "r"(mbar)
      : "memory");
}
// Operand descriptor in the 128-byte swizzle: 8 rows (K-major) or 8 k steps (N contiguous) of 128
// bytes to an atom, atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

template <bool F16>
struct Smem128 {
  static constexpr int kStages = F16 ? 2 : 1;
  uint4 ring[kStages][2][tile128(F16) * (F16 ? 8 : 16)];  // K, V as they are, at 1024 bytes
  uint4 tile[F16 ? 1 : 6][F16 ? 1 : kTile * 8];           // f32 cache: K hi, mid, lo, V hi, mid, lo
  float ex[2][128];                                // what a row's threads tell each other
  unsigned long long mbar[4];                      // s, o, a tile's copies in each stage
  unsigned long long bad;
  uint32_t tmem;
  Tile128 next[3];  // of tile i: i % 3
  Cursor pre;
  int t_begin;
  Plan plan;
};

template <bool F16>
__global__ void __launch_bounds__(kThreads128, 2)
    k_tree_attn_128(TreeAttnArgs a, const __grid_constant__ Maps128 maps) {
  using KV = typename std::conditional<F16, __half, float>::type;
  using S = Smem128<F16>;
  constexpr int BM = 128, kT = tile128(F16), NS = kT / 2, ND = kHd / 2;  // NS scores, ND dims to a thread
  constexpr int kParts = F16 ? 2 : 3;  // of q and p; of K and V one or three
  constexpr uint32_t kType = F16 ? 0 : kIdescBf16, kPartBytes = kTile * 128;
  // tensor memory: s (kT columns), for every 16 positions overlaid by 8 + 8 columns of p's first two
  // parts; the third part, 8 columns for every 16 positions; o; q, 16 columns a part for every 32 dims
  constexpr uint32_t kColsP = kT, kColsO = F16 ? kT : kT + kT / 2, kColsQ = kColsO + kHd, kCols128 = 256;
  static_assert(kColsQ + 32 * kParts <= kCols128, "tensor memory of half an SM");
  extern __shared__ __align__(128) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + (1024 - (tc::smem_u32(smem_raw) & 1023)) % 1024);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int lrow = tid & 127, half = tid >> 7;
  constexpr int kStepper = 128;  // the thread that steps through the units and copies; warp 0 issues the products
  const int uwarp = __shfl_sync(0xffffffffu, warp, 0);  // known to be the warp's: descriptors stay in uniform registers

  pdl_trigger();
  if (warp == 0) make_plan<-kT>(a, BM, &sm.plan);
  __syncthreads();
  int end;
  {
    Cursor cur;
    if (!first_tile<BM>(a, sm.plan, cur, end)) return;
    if (tid == kStepper) {
      sm.pre = cur;
      sm.t_begin = -1;
    }
  }
  // one thread: the tile at sm.pre, and on to the next
  auto step = [&](int i) {
    Tile128& n = sm.next[i % 3];
    Cursor c = sm.pre;
    n.valid = c.u < end;
    if (!n.valid) return;
    n.draft = c.t == c.nt - 1;
    const int row0 = n.draft ? 0 : c.t * kT;
    n.base = (c.head * (n.draft ? a.n_nodes : a.max_ctx) + row0) * kHd;
    n.left = c.p0 - row0;
    n.rows = n.draft ? c.cnt : min(kT, n.left);
    n.b = c.b;
    n.h = c.h;
    n.r = c.r;
    n.cnt = c.cnt;
    n.begin = sm.t_begin < 0;
    const int first = n.begin ? c.t : sm.t_begin;
    n.last = n.draft || c.u + 1 >= end;
    n.whole = first == 0 && n.draft;
    n.slot = first > 0 ? 0 : 1;
    sm.t_begin = n.last ? -1 : first;
    advance(sm.plan, a.n_kv, c);
    sm.pre = c;
  };
  if (tid == kStepper) {
    step(0);
    step(1);
  }

  const uint32_t mb_s = tc::smem_u32(&sm.mbar[0]), mb_o = tc::smem_u32(&sm.mbar[1]);
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&sm.tmem)),
                 "r"(kCols128)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    sm.bad = 0;
    tc::mbar_init(mb_s, 1);
    tc::mbar_init(mb_o, 1);
    tc::mbar_init(mb_o + 8, 1);
    tc::mbar_init(mb_o + 16, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = sm.tmem, mine = tm + ((uint32_t)(32 * (warp & 3)) << 16);  // this warp's lanes

  const KV* kc = static_cast<const KV*>(a.kc);
  const KV* vc = static_cast<const KV*>(a.vc);
  const KV* kd = static_cast<const KV*>(a.kd);
  const KV* vd = static_cast<const KV*>(a.vd);

  // One thread: copy tile i into its ring slot.  Binary16: whole boxes of 64 rows, whatever lies
  // behind the last one (its scores are masked, its values cleared below); f32: the rows that exist.
  auto produce = [&](int i) {
    const Tile128& n = sm.next[i % 3];
    if (!n.valid) return;
    const int slot = i % S::kStages;
    const uint32_t dk = tc::smem_u32(sm.ring[slot][0]), dv = tc::smem_u32(sm.ring[slot][1]), mb = mb_o + 8 + 8 * slot;
    if constexpr (F16) {
      const int boxes = n.draft ? 1 : kT / kBoxRows, row = (int)(n.base / kHd);
      tc::mbar_arrive_expect_tx(mb, 2u * boxes * kBoxRows * 128);
      for (int x = 0; x < boxes; ++x) {
        tma_rows(dk + x * kBoxRows * 128, &maps.m[n.draft ? 2 : 0], row + x * kBoxRows, mb);
        tma_rows(dv + x * kBoxRows * 128, &maps.m[n.draft ? 3 : 1], row + x * kBoxRows, mb);
      }
    } else {
      const uint32_t bytes = (uint32_t)n.rows * kHd * 4;
      tc::mbar_arrive_expect_tx(mb, 2 * bytes);
      tc::bulk_copy_g2s(dk, (n.draft ? kd : kc) + n.base, bytes, mb);
      tc::bulk_copy_g2s(dv, (n.draft ? vd : vc) + n.base, bytes, mb);
    }
  };
  if (tid == kStepper) {
    produce(0);
    if (F16) produce(1);
  }
  __syncwarp();

  // One thread: the products of the parts, the smallest first (what is cut off there does not
  // count): mul(part of the A operand, part of the B operand, 0 for the first one).
  auto products = [&](auto&& mul) {
    if constexpr (F16) {
      mul(1, 0, 0);
    } else {
      mul(2, 0, 0);
      mul(0, 2, 1);
      mul(1, 1, 1);
      mul(1, 0, 1);
      mul(0, 1, 1);
    }
    mul(0, 0, 1);
  };
  // s = q k^T
  auto issue_s = [&](uint32_t k) {
    tc::fence_after_sync();
    products([&](int a_part, int b_part, int more) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {  // 16 dims: 8 columns of q
        const uint32_t at = k + kPartBytes * b_part;
        tc::mma_f16_ts(tm, tm + kColsQ + 16 * (kParts * (ks / 2) + a_part) + 8 * (ks & 1),
                       F16 ? desc_sw128(at + 32 * ks) : tc::smem_desc(at + 256 * ks, 128, 1024),
                       tc::idesc_f16(128, kT) | kType, more || ks > 0);
      }
    });
  };

  float o[ND];
  float m = -INFINITY, l = 0.f, rs = 1.f;
  uint64_t vis = 0;
  bool lost = false;  // a wait has run out: the rows of the walk are NaN

  int it = 0;
  for (; sm.next[it % 3].valid; ++it) {
    const Tile128& cur = sm.next[it % 3];
    const bool draft = cur.draft;
    const int rows = cur.cnt * a.group;
    const int row = cur.r * BM + lrow;
    const bool warp_live = cur.r * BM + 32 * (warp & 3) < rows;
    if (cur.begin) {
      // the last walk's products are done (every thread has waited for its o): q may change
      const bool live = row < rows;
      const float* src = row_of(a, const_cast<float*>(a.q), cur, live ? row : 0);
      src += (int64_t)cur.b * (a.q_batch_stride - (int64_t)a.n_nodes * a.n_kv * a.group * kHd) + half * ND;
      float4 x[8];
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        x[c] = live ? __ldcg(reinterpret_cast<const float4*>(src) + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float scale = 1.4426950408889634f * 0.125f;  // scores in log2 units
        x[c].x *= scale;
        x[c].y *= scale;
        x[c].z *= scale;
        x[c].w *= scale;
        mx = max(mx, abs_max(x[c]));
      }
      vis = live ? a.mask[(int64_t)cur.b * a.n_nodes + row / a.group] : 0ull;
      if (cur.cnt < 64) vis &= (1ull << cur.cnt) - 1;
      float f = 1.f;
      if constexpr (F16) {
        sm.ex[half][lrow] = __uint_as_float(mx);
        __syncthreads();
        const int e = scale_exp(max(mx, __float_as_uint(sm.ex[half ^ 1][lrow])));
        rs = pow2(e);
        f = pow2(-e);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t part[kParts][8];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const float4 y = x[4 * c + d / 2];
          float2 z = d & 1 ? make_float2(y.z * f, y.w * f) : make_float2(y.x * f, y.y * f);
          if constexpr (F16) {
            split2(z.x, z.y, part[0][d], part[1][d]);
          } else {
#pragma unroll
            for (int p = 0; p < kParts; ++p) part[p][d] = bf16_part(z);
          }
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p) tmem_st8(mine + kColsQ + 16 * (kParts * half + p) + 8 * c, part[p]);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      m = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] = 0.f;
    }

    // ---- the tile arrives
    const int slot = it % S::kStages;
    const uint32_t mb_full = mb_o + 8 + 8 * slot, full = (uint32_t)(it / S::kStages) & 1u;
    uint32_t k_at, v_at;  // the first parts
    if constexpr (F16) {
      k_at = tc::smem_u32(sm.ring[slot][0]);
      v_at = tc::smem_u32(sm.ring[slot][1]);
      if (cur.rows < kT) {
        // Behind the last row lies what the cache happens to hold, and a draft's values may hold
        // an infinity or NaN: either would reach every row of the product (0 times it is NaN).
        // Such rows are cleared here; a draft's is added below where it is seen.
        if (!lost && !tc::mbar_wait(mb_full, full)) lost = true;
        for (int r = tid >> 2; r < kT; r += kThreads128 / 4) {
          uint4* v = sm.ring[slot][1] + r * 8 + (tid & 3) * 2;
          uint32_t off = 0;
          if (draft && r < cur.rows) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint4 w = v[c];
              off |= (((w.x & 0x7C007C00u) + 0x04000400u) | ((w.y & 0x7C007C00u) + 0x04000400u) |
                      ((w.z & 0x7C007C00u) + 0x04000400u) | ((w.w & 0x7C007C00u) + 0x04000400u)) &
                     0x80008000u;
            }
          }
          off |= __shfl_xor_sync(0xffffffffu, off, 1);
          off |= __shfl_xor_sync(0xffffffffu, off, 2);
          if (off && !(tid & 3)) atomicOr(&sm.bad, 1ull << r);
          if (off || r >= cur.rows) v[0] = v[1] = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
      }
    } else {
      if (!lost && !tc::mbar_wait(mb_full, full)) lost = true;
      // four threads to a position, 16 dims each; their 16-byte reads in an order without bank
      // conflicts
      const int r = tid >> 2, j = tid & 3, turn = (j >> 1) + 2 * (r & 1);
      const float4* kraw = reinterpret_cast<const float4*>(sm.ring[0][0]) + r * 16 + 4 * j;
      const float4* vraw = reinterpret_cast<const float4*>(sm.ring[0][1]) + r * 16 + 4 * j;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = r < cur.rows ? (kv ? vraw : kraw)[i ^ turn] : make_float4(0.f, 0.f, 0.f, 0.f);
        if (kv && draft) {  // a row that has no bfloat16 parts, cleared as above
          uint32_t mx = max(max(abs_max(x[0]), abs_max(x[1])), max(abs_max(x[2]), abs_max(x[3])));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          if (mx >= kFarBits) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j == 0) atomicOr(&sm.bad, 1ull << r);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 lo = make_float2(x[i].x, x[i].y), hi = make_float2(x[i].z, x[i].w);
          const int c = 4 * j + (i ^ turn);
          const uint32_t at = core_off(r, c >> 1) / 8 + (c & 1);
#pragma unroll
          for (int p = 0; p < 3; ++p)
            reinterpret_cast<uint2*>(sm.tile[3 * kv + p])[at] = make_uint2(bf16_part(lo), bf16_part(hi));
        }
      }
      k_at = tc::smem_u32(sm.tile[0]);
      v_at = tc::smem_u32(sm.tile[3]);
    }

    // ---- scores (of a binary16 tile inside a walk they were issued behind the last tile's products)
    if (!F16 || cur.begin) {
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncthreads();
      if (F16 && uwarp == 0 && !lost && !tc::mbar_wait(mb_full, full)) lost = true;
      __syncwarp();
      if (uwarp == 0 && elect_one()) {
        issue_s(k_at);
        tc::mma_commit(mb_s);
      }
      __syncwarp();
      if (!F16 && tid == kStepper) produce(it + 1);  // all threads have read the raw tile
      __syncwarp();
    }
    if (!lost && !tc::mbar_wait(mb_s, (uint32_t)it & 1u)) lost = true;
    tc::fence_after_sync();

    // 16 or 32 of this thread's scores, in log2 units but for the row's scale; what the row does not
    // see is -INFINITY
    const bool partial = draft || cur.left < kT;
    uint64_t see = ~0ull;
    if (partial) {
      const int in = min(max(cur.left - NS * half, 0), 64);
      see = draft ? (half * NS < 64 ? vis >> (half * NS & 63) : 0ull) : in < 64 ? (1ull << in) - 1 : ~0ull;
    }
    auto scores = [&](int c, auto& s) {
      constexpr int n = sizeof(s) / 4;
      if constexpr (n == 16)
        tmem_ld16(mine + NS * half + 16 * c, s);
      else
        tc::tmem_ld32(mine + NS * half + 16 * c, s);
      if (partial) {
        const uint32_t bits = (uint32_t)(see >> (16 * c));
#pragma unroll
        for (int j = 0; j < n; ++j)
          if (!(bits >> j & 1)) s[j] = -INFINITY;
      }
    };
    float corr = 1.f;
    if (warp_live) {
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < NS / 32; ++c) {
        float s[32];
        scores(2 * c, s);
#pragma unroll
        for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], s[j]);
      }
      sm.ex[half][lrow] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * rs;
    }
    __syncthreads();  // the maximum of the row's other half
    if (warp_live) {
      // ---- online softmax
      const float mn = fmaxf(m, fmaxf(sm.ex[0][lrow], sm.ex[1][lrow]));
      const float mu = mn == -INFINITY ? 0.f : mn;
      corr = ex2(m - mu);
      m = mn;
      const float bias = (F16 ? kBias : 0.f) - mu;
      float2 sum = make_float2(0.f, 0.f), sum1 = sum;
#pragma unroll
      for (int c = 0; c < NS / 16; ++c) {
        float s[16];
        scores(c, s);
        // ---- the weights' parts over the scores
        uint32_t part[kParts][8];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float2 p = fma2(make_float2(s[j], s[j + 1]), make_float2(rs, rs), make_float2(bias, bias));
          p.x = ex2(p.x);
          p.y = ex2(p.y);
          if (j & 2)
            sum1 = add2(sum1, p);
          else
            sum = add2(sum, p);
          if constexpr (F16) {
            const __half2 h = __floats2half2_rn(p.x, p.y);
            const float2 back = __half22float2(h);
            const float2 rest = fma2(back, make_float2(-1.f, -1.f), p);
            const __half2 w = __floats2half2_rn(rest.x, rest.y);
            part[0][j / 2] = *reinterpret_cast<const uint32_t*>(&h);
            part[1][j / 2] = *reinterpret_cast<const uint32_t*>(&w);
          } else {
#pragma unroll
            for (int x = 0; x < kParts; ++x) part[x][j / 2] = bf16_part(p);
          }
        }
        tmem_st8(mine + NS * half + 16 * c, part[0]);
        tmem_st8(mine + NS * half + 16 * c + 8, part[1]);
        if constexpr (!F16) tmem_st8(mine + kColsP + NS / 2 * half + 8 * c, part[2]);
      }
      l = fmaf(l, corr, (sum.x + sum.y) + (sum1.x + sum1.y));
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
    const unsigned long long bad = draft ? sm.bad : 0ull;
    if (bad) {
      if (vis & bad) {  // the other rows keep every bit
        const int64_t at = ((int64_t)cur.b * a.n_kv + cur.h) * a.n_nodes * kHd;
        const float* qrow = row_of(a, const_cast<float*>(a.q), cur, row) +
                            (int64_t)cur.b * (a.q_batch_stride - (int64_t)a.n_nodes * a.n_kv * a.group * kHd);
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= corr;
        corr = 1.f;
        for (int j = 0; j < kTile; ++j) {
          if (!((vis & bad) >> j & 1)) continue;
          float x = 0.f;
          for (int d = 0; d < kHd; ++d) x = fmaf(qrow[d], (float)kd[at + j * kHd + d], x);
          const float p =
              ex2(fmaf(x, 1.4426950408889634f * 0.125f, (F16 ? kBias : 0.f) - (m == -INFINITY ? 0.f : m)));
#pragma unroll
          for (int d = 0; d < ND; ++d) o[d] += p * (float)vd[at + j * kHd + half * ND + d];
        }
      }
    }
    tc::fence_before_sync();
    __syncthreads();

    // ---- weighted values
    if (uwarp == 0 && elect_one()) {
      tc::fence_after_sync();
      products([&](int a_part, int b_part, int more) {
#pragma unroll
        for (int kk = 0; kk < kT / 16; ++kk) {  // 16 positions: 8 columns of p, two atoms or rows of core matrices of v
          const uint32_t p = a_part < 2 ? tm + 16 * kk + 8 * a_part : tm + kColsP + 8 * kk;
          const uint32_t at = v_at + kPartBytes * b_part + 2048 * kk;
          tc::mma_f16_ts(tm + kColsO, p, F16 ? desc_sw128(at) : tc::smem_desc(at, 1024, 128), kIdescO | kType,
                         more || kk > 0);
        }
      });
      tc::mma_commit(mb_o);
    }
    __syncwarp();  // no lane polls while another of its warp still has the products to issue
    if (tid == kStepper) step(it + 2);  // over tile it - 1's, which everyone is done with
    __syncwarp();
    if (!lost && !tc::mbar_wait(mb_o, (uint32_t)it & 1u)) lost = true;
    if constexpr (F16) {
      // p and this tile's slot are read: the next tile's scores, under the sums below, and the
      // copy of the one after it
      if (uwarp == 0) {
        const bool ahead = sm.next[(it + 1) % 3].valid && !sm.next[(it + 1) % 3].begin;
        const int ns = (it + 1) % S::kStages;
        if (ahead && !lost && !tc::mbar_wait(mb_o + 8 + 8 * ns, (uint32_t)((it + 1) / S::kStages) & 1u))
          lost = true;
        __syncwarp();
        if (ahead && elect_one()) {
          issue_s(tc::smem_u32(sm.ring[ns][0]));
          tc::mma_commit(mb_s);
        }
      }
      if (tid == kStepper) produce(it + 2);
      __syncwarp();
    }
    tc::fence_after_sync();
    if (warp_live) {
#pragma unroll
      for (int d0 = 0; d0 < ND; d0 += 16) {
        float t[16];
        tmem_ld16(mine + kColsO + ND * half + d0, t);
#pragma unroll
        for (int d = 0; d < 16; d += 2) {
          const float2 x =
              fma2(make_float2(o[d0 + d], o[d0 + d + 1]), make_float2(corr, corr), make_float2(t[d], t[d + 1]));
          o[d0 + d] = x.x;
          o[d0 + d + 1] = x.y;
        }
      }
    }

    // ---- the end of this CTA's part of the walk
    if (cur.last) {
      const bool whole = cur.whole;
      if (__syncthreads_or(lost)) l = NAN;  // every thread has read `bad` and `ex`
      sm.ex[half][lrow] = l;
      if (tid == 0) sm.bad = 0;
      __syncthreads();
      const float lt = l + sm.ex[half ^ 1][lrow];
      float* part = a.ws + ((int64_t)blockIdx.x * 2 + cur.slot) * part_floats(BM);
      if (!whole && half == 0) {
        part[lrow] = m;
        part[BM + lrow] = lt;
      }
      if (!whole || row < rows) {
        const float inv = !whole ? 1.f : lt == 0.f ? 0.f : 1.f / lt;
        float4* dst = reinterpret_cast<float4*>((whole ? row_of(a, a.out, cur, row) : part + 2 * BM + lrow * kHd) +
                                                half * ND);
        const bool none = whole && lt == 0.f;
#pragma unroll
        for (int d = 0; d < ND; d += 4)
          dst[d / 4] = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(o[d] * inv, o[d + 1] * inv, o[d + 2] * inv, o[d + 3] * inv);
      }
      __syncthreads();  // `ex` is read
    }
  }
  tc::fence_before_sync();
  if (__syncthreads_or(lost) && tid == kStepper) {  // products and copies that nobody waited for
    tc::mbar_wait(mb_o, (uint32_t)(it - 1) & 1u);
    for (int x = 0; x < min(it, S::kStages); ++x)
      tc::mbar_wait(mb_o + 8 + 8 * x, (uint32_t)((it - 1 - x) / S::kStages) & 1u);
  }
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kCols128) : "memory");
}

// Joins the parts of the walks that more than one CTA took: block x the walk, if any, whose first
// tile is CTA x's and whose last is not, a warp to a row.  A walk of many parts has the blocks of
// its next three CTAs as well, a block to a row and a quarter of the parts to a warp.  Also the
// zeros of the sequences whose position is out of range.
// Bound by the latency of the loads (L2), so those of kJoin parts are under way together.  One
// kv head, 15 rows, 16000 / 64000 positions binary16: 8.3 / 15.6 us the whole call, 11.6 / 29.0 with a
// warp to a row whatever the parts, 13.8 / 37.9 with 4 parts at once (16 at once: 8.0 / 16.1, but
// 65 against 59 us for 64 x 32 rows of 32700 positions).  kFewParts 8 instead of 16: 8.5 against 9.0 us
// for 32 rows of 4000 positions, 36.3 against 33.7 us for 8 x 512 rows of 4000, whose blocks would
// be four times as many.
constexpr int kRows = kThreads / 32;  // of a block
constexpr int kFewParts = 16, kJoin = 8;
template <int BM, int SUB>
__global__ void __launch_bounds__(kThreads) k_tree_attn_join(TreeAttnArgs a, int ctas) {
  __shared__ Plan plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) make_plan<SUB>(a, BM, &plan);
  __syncthreads();
  pdl_wait();  // in every CTA: the end of this kernel is the end of both
  const int first = blockIdx.x;
  if (first < a.batch && !plan.nt[first]) {
    const int64_t n = (int64_t)plan.cnt[first] * a.n_kv * a.group * (kHd / 4);
    float4* z = reinterpret_cast<float4*>(a.out + (int64_t)first * a.n_nodes * a.n_kv * a.group * kHd);
    for (int64_t x = (int64_t)blockIdx.y * kThreads + threadIdx.x; x < n; x += (int64_t)gridDim.y * kThreads)
      z[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int total = plan.off[QD_MAX_BATCH], per = units_per_cta(total, ctas);
  if ((int64_t)first * per >= total) return;
  const int last_unit = min((int64_t)(first + 1) * per, (int64_t)total) - 1;
  Cursor cur;  // the walk of this CTA's last unit
  cur.b = 0;
  while (last_unit >= plan.off[cur.b + 1]) ++cur.b;
  const int nt = plan.nt[cur.b], walk = (last_unit - plan.off[cur.b]) / (nt + kStart);
  cur.h = walk / plan.rb[cur.b];
  cur.r = walk % plan.rb[cur.b];
  const int g0 = plan.off[cur.b] + walk * (nt + kStart) + kStart;  // its first tile's unit
  const int c0 = g0 / per, c1 = (g0 + nt - 1) / per;
  const bool few = c1 - c0 < kFewParts;
  const int x = first - c0;  // -1: the last unit is of the walk's start, before its first tile
  if (c0 == c1 || x < 0 || x >= (few ? 1 : kRows)) return;
  const int r = blockIdx.y * kRows + (few ? warp : x), at = cur.r * BM + r;
  if (at >= plan.cnt[cur.b] * a.group) return;
  float m = -INFINITY, l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  auto join = [&](const float (&mc)[kJoin], const float (&lc)[kJoin], const float2 (&oc)[kJoin]) {
    float top = m;
#pragma unroll
    for (int i = 0; i < kJoin; ++i) top = fmaxf(top, mc[i]);
    const float f = m == -INFINITY ? l : ex2(m - top);  // without a maximum l is 0 or NaN
    m = top;
    l *= f;
    o.x *= f;
    o.y *= f;
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      const float g = mc[i] == -INFINITY ? lc[i] : ex2(mc[i] - top);
      l = fmaf(lc[i], g, l);
      o.x = fmaf(oc[i].x, g, o.x);
      o.y = fmaf(oc[i].y, g, o.y);
    }
  };
  const int step = few ? 1 : kRows;
  for (int c = few ? c0 : c0 + warp; c <= c1; c += step * kJoin) {
    float mc[kJoin], lc[kJoin];
    float2 oc[kJoin];
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      const int at_c = c + i * step;
      // the walk begins in its first CTA (slot 1: that CTA's last part) and is the first part of the others
      const float* p = a.ws + ((int64_t)at_c * 2 + (at_c == c0 ? 1 : 0)) * part_floats(BM);
      const bool live = at_c <= c1;
      mc[i] = live ? __ldcg(p + r) : -INFINITY;
      lc[i] = live ? __ldcg(p + BM + r) : 0.f;
      oc[i] = live ? __ldcg(reinterpret_cast<const float2*>(p + 2 * BM + r * kHd) + lane) : make_float2(0.f, 0.f);
    }
    join(mc, lc, oc);
  }
  if (!few) {  // the warps' quarters
    static_assert(kJoin >= kRows, "joined at once");
    __shared__ float ms[kRows], ls[kRows];
    __shared__ float2 os[kRows][32];
    os[warp][lane] = o;
    if (lane == 0) {
      ms[warp] = m;
      ls[warp] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    float mc[kJoin], lc[kJoin];
    float2 oc[kJoin];
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      mc[i] = i < kRows ? ms[i] : -INFINITY;
      lc[i] = i < kRows ? ls[i] : 0.f;
      oc[i] = i < kRows ? os[i][lane] : make_float2(0.f, 0.f);
    }
    m = -INFINITY;
    l = 0.f;
    o = make_float2(0.f, 0.f);
    join(mc, lc, oc);
  }
  reinterpret_cast<float2*>(row_of(a, a.out, cur, at))[lane] =
      l == 0.f ? make_float2(0.f, 0.f) : make_float2(o.x / l, o.y / l);
}

// Blocks of 16 rows or of 128.  Up to 32 rows to a kv head 16 (two blocks; 54.9 us for 32 rows at
// 4000 positions of 2 x 32 heads f32, where 128-row blocks take 61.7 us whatever they hold).  More
// rows are walks by the dozen in blocks of 16, which read a head's positions once each; that fills
// the SMs while there is little work, and a walk starts in fewer steps.  The work is counted in
// positions of a 16-row block as the cache has room for, a start as 1000 of them.  16 against 128
// rows, in us, one sequence:
//   f32       8 x 64 rows, 500 positions (work 50e3)      12.0 13.6
//             4 x 128, 2000 (98e3)                         15.2 15.6
//             9 x 40, 3000, two sequences (221e3)          25.4 27.8
//             3 x 36, 8000, three sequences (246e3)        27.3 29.9
//             1 x 216, 3000, five ragged ones (280e3)      17.9 19.7
//             4 x 128, 8000 (291e3)                        32.3 26.6
//             4 x 512, 2000 (396e3)                        34.5 27.9
//             8 x 512, 8000 (2.3e6)                       189.9 67.7
// (on f32 caches rows that fill their blocks of 128 gain from half the bound on, those that do not
// from above it on)
//   binary16  8 x 64, 500 (50e3)                           10.5 14.9
//             8 x 256, 2000 (392e3)                        19.5 23.0
//             4 x 512, 8000 (1.16e6)                       40.5 33.3
//             1 x 512, 32000 (1.06e6)                      39.9 41.4
//             8 x 512, 8000 (2.3e6)                        70.5 42.7
constexpr int64_t kWork16 = 300000, kWork16F16 = 1100000;
inline bool by16(int n_kv, int group, int n_nodes, int max_ctx, int batch, bool f16) {
  const int blocks = (n_nodes * group + 15) / 16;
  return blocks <= 2 || (int64_t)batch * n_kv * blocks * ((int64_t)max_ctx + 1000) <= (f16 ? kWork16F16 : kWork16);
}
inline int blocks_of(int n_nodes, int group, int bm) { return (n_nodes * group + bm - 1) / bm; }
constexpr int kMaxCtas = 2;  // CTAs to an SM at most
// CTAs of a call: what fits the device at once, and no more than there can be units for.
inline int tree_ctas(int n_kv, int blocks, int n_nodes, int max_ctx, int batch, int sub, int per_sm) {
  const int64_t units = (int64_t)batch * n_kv * blocks * (walk_tiles(sub, max_ctx, n_nodes) + kStart);
  return (int)std::min<int64_t>((int64_t)attn_sm_count() * per_sm, (units + kMinPer - 1) / kMinPer);
}

template <int BM, int SUB, typename... More>
qd_status launch(const TreeAttnArgs& a, void (*kern)(TreeAttnArgs, More...), int threads, size_t smem, int per_sm,
                 cudaStream_t st, const std::remove_const_t<More>&... more) {
  static std::atomic<bool> done[64];  // one kernel to an instance of this function
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QD_ERR_CUDA;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return QD_ERR_CUDA;
    done[dev] = true;
  }
  const int walks = a.batch * a.n_kv * a.blocks;
  const int ctas = a.whole ? walks : tree_ctas(a.n_kv, a.blocks, a.n_nodes, a.max_ctx, a.batch, SUB, per_sm);
  kern<<<ctas, threads, smem, st>>>(a, more...);
  const qd_status s = launch_status();
  if (s != QD_OK || a.whole) return s;
  return launch_k(k_tree_attn_join<BM, SUB>, dim3((unsigned)ctas, BM / 4), dim3(kThreads), 0, st, true, a, ctas);
}

// The map of `rows` rows of 64 binary16 values, in boxes of kBoxRows.
bool row_map(CUtensorMap* map, const void* base, int64_t rows) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[2] = {kHd, (cuuint64_t)rows}, strides[1] = {kHd * 2};
  const cuuint32_t box[2] = {kHd, kBoxRows}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F16>
qd_status launch_f(const TreeAttnArgs& a, bool rows16, cudaStream_t st) {
  if (rows16)
    return launch<16, sub_positions(F16)>(a, k_tree_attn_16<F16>, Smem16<F16>::kWarps * 32, sizeof(Smem16<F16>), 2, st);
  Maps128 maps = {};
  if constexpr (F16) {
    const int64_t heads = (int64_t)a.batch * a.n_kv;
    const void* base[4] = {a.kc, a.vc, a.kd, a.vd};
    for (int i = 0; i < 4; ++i)
      if (!row_map(&maps.m[i], base[i], heads * (i < 2 ? a.max_ctx : a.n_nodes))) return QD_ERR_CUDA;
  }
  return launch<128, -tile128(F16)>(a, k_tree_attn_128<F16>, kThreads128, sizeof(Smem128<F16>) + 1024, 2, st, maps);
}

// The units of a call must fit an int.
inline bool tree_shape_ok(int n_heads, int n_kv_heads, int head_dim, int n_nodes, int max_ctx, int batch) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > 8 || head_dim != kHd ||
      n_nodes < 1 || n_nodes > QD_MAX_TREE || max_ctx < 1 || batch < 1 || batch > QD_MAX_BATCH)
    return false;
  // (blocks of 16 with more than 32 rows: by16 keeps their work far below this)
  const int rows = n_nodes * (n_heads / n_kv_heads);
  const int64_t walks = (int64_t)batch * n_kv_heads * ((rows + 127) / 128 + (rows > 16 && rows <= 32));
  if ((int64_t)batch * n_kv_heads * std::max(max_ctx, n_nodes) > (1ll << 31) - 128) return false;  // rows of a cache
  return walks <= (1 << 20) && walks * ((int64_t)max_ctx / kTile + 2 + kStart) <= (1 << 30);
}

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

size_t qd_tree_attn_workspace(int n_heads, int n_kv_heads, int head_dim, int n_nodes, int max_ctx, int batch) {
  if (!tree_shape_ok(n_heads, n_kv_heads, head_dim, n_nodes, max_ctx, batch)) return 0;
  const int group = n_heads / n_kv_heads;
  size_t most = 0;  // of either cache type
  for (const bool f16 : {false, true}) {
    const bool rows16 = by16(n_kv_heads, group, n_nodes, max_ctx, batch, f16);
    const int bm = rows16 ? 16 : 128;
    const int ctas = tree_ctas(n_kv_heads, blocks_of(n_nodes, group, bm), n_nodes, max_ctx, batch,
                               rows16 ? sub_positions(f16) : -tile128(f16), kMaxCtas);
    most = std::max(most, (size_t)ctas * 2 * part_floats(bm) * sizeof(float));
  }
  return most;
}

qd_status qd_tree_attn(const float* q, int64_t q_batch_stride, const void* k_cache, const void* v_cache,
                       const void* k_draft, const void* v_draft, int kv_f16, float* out, int n_heads, int n_kv_heads,
                       int head_dim, const int32_t* pos, const uint64_t* mask, const int32_t* n_valid, int n_nodes,
                       int max_ctx, int batch, void* workspace, size_t workspace_bytes, qd_stream_t stream) {
  if (!q || !k_cache || !v_cache || !k_draft || !v_draft || !out || !pos || !mask || !workspace)
    return QD_ERR_INVALID_ARG;
  if (kv_f16 != 0 && kv_f16 != 1) return QD_ERR_INVALID_ARG;
  if (head_dim != kHd) return QD_ERR_UNSUPPORTED;
  const size_t need = qd_tree_attn_workspace(n_heads, n_kv_heads, head_dim, n_nodes, max_ctx, batch);
  if (!need) return QD_ERR_SHAPE;
  if (batch > 1 && q_batch_stride < (int64_t)n_nodes * n_heads * head_dim) return QD_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_draft) || !aligned16(v_draft) ||
      !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(mask) & 7) ||
      ((reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(n_valid)) & 3))
    return QD_ERR_ALIGN;
  if (batch > 1 && q_batch_stride % 4) return QD_ERR_ALIGN;
  if (workspace_bytes < need) return QD_ERR_NOMEM;
  TreeAttnArgs a;
  a.q = q;
  a.q_batch_stride = q_batch_stride;
  a.kc = k_cache;
  a.vc = v_cache;
  a.kd = k_draft;
  a.vd = v_draft;
  a.out = out;
  a.n_kv = n_kv_heads;
  a.group = n_heads / n_kv_heads;
  a.pos = pos;
  a.mask = mask;
  a.n_valid = n_valid;
  a.n_nodes = n_nodes;
  a.max_ctx = max_ctx;
  a.batch = batch;
  a.ws = static_cast<float*>(workspace);
  const bool rows16 = by16(n_kv_heads, a.group, n_nodes, max_ctx, batch, kv_f16);
  a.blocks = blocks_of(n_nodes, a.group, rows16 ? 16 : 128);
  const int sub = rows16 ? sub_positions(kv_f16) : -tile128(kv_f16);
  a.whole = walk_tiles(sub, max_ctx, n_nodes) <= kWholeTiles;
  return kv_f16 ? launch_f<true>(a, rows16, (cudaStream_t)stream) : launch_f<false>(a, rows16, (cudaStream_t)stream);
}

}  // extern "C"
