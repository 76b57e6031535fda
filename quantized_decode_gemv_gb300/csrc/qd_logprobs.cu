// Log probabilities of given tokens, entropy and the top alternatives of rows of logits.
// With m = max x, and r and h the sums of e^(x - m) and e^(x - m) (x - m) over all values but
// one largest,
//   log p_t = (x_t - m) - log1p(r)
//   H       = log1p(r) - h / (1 + r)
// Both terms of H are positive and r leaves the largest out, so neither loses digits when one
// token holds nearly all of the probability.  Parts (m, r, h) join as
//   (1 + r_a) e^(m_a - m) and (h_a + (m_a - m) (1 + r_a)) e^(m_a - m).
//
// HBM bounds the call: 4 bytes and about eight instructions a value.  Rows stream through
// registers (two batches of two 16-byte loads a thread, no barrier) into a running (m, r, h) per
// thread, rescaled at most once per batch.  A row goes to one CTA, or to a cluster of up to 8
// where there are few rows.  At the end of the row:
//  1. the k-th largest of the 256 threads' maxima (a bitonic sort per warp, joined by one warp)
//     is at most the slice's k-th largest value.  The values of the threads whose maximum
//     reaches that bound, k of them, are read again (from L2, a warp to a thread's values) and
//     those that reach it listed, k and few more; with them the sums of one thread that holds a
//     largest value, to leave that one out.  A list that overflows (many equal values) falls
//     back to the values above the bound and an ordered scan for those equal to it;
//  2. the list is ranked by counting, the slices' results go through distributed shared memory
//     to the cluster's first CTA, whose first warp joins them.
// Measured (one GB300, 2048 rows of 49152, top 5): 71 us, 5.7 TB/s of 6.8 (a plain read of as
// many bytes: 61 us); 8 CTAs to an SM with 2 + 2 loads against 4 with 4 + 4: 71 against 77 us, and
// 11.8 against 17.6 us for 2048 rows of 1000.  With the slices in shared memory and the sums
// behind a barrier it took 174 us (a CTA's phases follow one another and its loads wait for the
// slowest), with every thread reading its own values again 100 us.
// No atomic's order shows: the list is ranked by (value, index), sums have a fixed order.
#include <cooperative_groups.h>

#include "qd_internal.cuh"

namespace qd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 256;           // values at or above the bound that are ranked at once
constexpr int kMaxSplit = 8;         // CTAs to a row
constexpr int kBatch = 2;            // 16-byte chunks that a thread loads at once
static_assert(QD_MAX_TOP == 32, "a warp holds a list of the largest");

typedef unsigned long long u64;

// Order of the values as an integer: larger value first, then the lower index; +0 and -0 are
// equal, and NaN stands behind everything.
__device__ __forceinline__ u64 order_key(float v, int i) {
  return v != v ? (u64)(0xFFFFFFFFu - (uint32_t)i) : argmax_key(v + 0.f, (uint32_t)i);
}
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return u == 0 ? NAN : __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 32 values, falling from lane 0 on.
__device__ __forceinline__ float sort_step(float v, int o, bool up, int lane) {
  const float w = __shfl_xor_sync(0xffffffffu, v, o);
  return ((lane & o) == 0) != up ? fmaxf(v, w) : fminf(v, w);
}
__device__ __forceinline__ float warp_sort(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) v = sort_step(v, o, size < 32 && (lane & size), lane);
  return v;
}
// The 32 largest of two falling lists, falling; `reversed` is the second one, rising.
__device__ __forceinline__ float warp_merge(float a, float reversed, int lane) {
  float v = fmaxf(a, reversed);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = sort_step(v, o, false, lane);
  return v;
}
__device__ __forceinline__ u64 warp_merge(u64 a, u64 reversed, int lane) {
  u64 v = a > reversed ? a : reversed;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 w = __shfl_xor_sync(0xffffffffu, v, o);
    v = (v > w) == ((lane & o) == 0) ? v : w;
  }
  return v;
}

struct Part {
  float m, r, h;
};
struct Shared {
  float wmax[kWarps][32];
  Part warp[kWarps];
  u64 list[kList];
  u64 top[QD_MAX_TOP];   // the slice's largest, falling; 0: none
  float bound;
  float2 own;            // sums of the thread that leaves a largest value out
  int count, owner, reached;
  uint8_t reach[kThreads];  // threads whose maximum reaches the bound
  // of the cluster's slices, in its first CTA
  Part parts[kMaxSplit];
  u64 tops[kMaxSplit][QD_MAX_TOP];
};

struct Args {
  const float* logits;
  int64_t row_stride;
  int vocab;
  const int32_t* tokens;
  int n_tokens;
  float *logprob, *entropy;
  int top_k;
  int32_t* top_idx;
  float* top_logprob;
  int chunks;  // 16-byte chunks of a slice
  int split;   // log2 of the CTAs to a row
};

// The slice: chunk c of the row's 16-byte aligned span holds values 4 c - lead .. 4 c - lead + 3;
// this CTA has chunks [c0, c0 + n).  What lies outside the row reads as -INFINITY.
struct Slice {
  const float* row;
  int vocab, lead, c0, n;
  __device__ __forceinline__ int index(int c) const { return 4 * (c0 + c) - lead; }
  __device__ __forceinline__ float at(int i) const { return i >= 0 && i < vocab ? __ldcg(row + i) : -INFINITY; }
  __device__ __forceinline__ float4 read(int c) const {
    const int i = index(c);
    if (i >= 0 && i + 3 < vocab) return __ldcg(reinterpret_cast<const float4*>(row + i));
    return make_float4(at(i), at(i + 1), at(i + 2), at(i + 3));
  }
};

// A thread's values so far: the largest, and the sums of e^(x - mu) and e^(x - mu) (x - mu)
// with mu = max(m, -FLT_MAX), so that rows of -INFINITY alone give sums of zero.
constexpr float kLowest = -3.402823466e38f;
struct Running {
  float m, r, h;
  __device__ __forceinline__ void add(float v, float mu) {
    const float d = max_nan(v - mu, -1e4f);  // finite: 0 times it is 0
    const float p = ex2(d * 1.4426950408889634f);
    r += p;
    h = fmaf(p, d, h);
  }
  __device__ __forceinline__ void raise(float to) {  // m becomes `to` > m
    const float d = max_nan(fmaxf(m, kLowest) - fmaxf(to, kLowest), -1e4f), f = ex2(d * 1.4426950408889634f);
    h = f * fmaf(d, r, h);
    r *= f;
    m = to;
  }
  __device__ __forceinline__ void add(const float4 (&x)[kBatch]) {
    float top = m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) top = fmaxf(fmaxf(fmaxf(top, x[j].x), fmaxf(x[j].y, x[j].z)), x[j].w);
    if (top > m) raise(top);
    const float mu = fmaxf(m, kLowest);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      add(x[j].x, mu);
      add(x[j].y, mu);
      add(x[j].z, mu);
      add(x[j].w, mu);
    }
  }
};

// Ranks the list's n keys by counting and stores the k largest in order.
__device__ __forceinline__ void rank_list(const u64* list, int n, int k, u64* top) {
  const int t = threadIdx.x;
  if (t < n) {
    const u64 mine = list[t];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > mine;
    if (rank < k) top[rank] = mine;
  }
}

// Appends, in rising index order, the values of the slice for which `pred` holds, until top
// holds k.  One warp.
template <typename P>
__device__ int scan_fill(const Slice& s, int have, int k, u64* top, P pred) {
  const int lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < 4 * s.n && have < k; e0 += 32) {
    const int e = e0 + lane, i = 4 * s.c0 - s.lead + e;
    const bool in = e < 4 * s.n && i >= 0 && i < s.vocab;
    const float v = in ? s.at(i) : 0.f;
    const bool hit = in && pred(v);
    const unsigned b = __ballot_sync(0xffffffffu, hit);
    const int at = have + __popc(b & ((1u << lane) - 1));
    if (hit && at < k) top[at] = order_key(v, i);
    have = min(k, have + __popc(b));
  }
  return have;
}

// Rare: too many values at the bound, or a slice with fewer than k numbers.  Takes the values
// above the bound, then those equal to it in order, then NaN in order.  If even those above
// overflow the list, one pass over the slice for each of the k largest.
__device__ __noinline__ void select_slow(const Slice& s, float bound, int k, Shared& sh) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) sh.count = 0;
  __syncthreads();
  for (int c = tid; c < s.n; c += kThreads) {
    const float4 x = s.read(c);
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v[j] > bound) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kList) sh.list[at] = order_key(v[j], s.index(c) + j);
      }
  }
  __syncthreads();
  const int n = sh.count;
  if (n <= kList) {
    rank_list(sh.list, n, k, sh.top);
    __syncthreads();
    if (tid < 32) {
      int have = scan_fill(s, min(n, k), k, sh.top, [bound](float v) { return v == bound; });
      if (have < k) scan_fill(s, have, k, sh.top, [](float v) { return v != v; });
    }
    __syncthreads();
    return;
  }
  u64 last = ~0ull;
  for (int r = 0; r < k; ++r) {
    u64 best = 0;
    for (int c = tid; c < s.n; c += kThreads) {
      const float4 x = s.read(c);
      const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = s.index(c) + j;
        const u64 key = order_key(v[j], i);
        if (i >= 0 && i < s.vocab && key < last && key > best) best = key;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const u64 other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    if ((tid & 31) == 0) sh.list[tid >> 5] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = sh.list[w] > best ? sh.list[w] : best;
    if (tid == 0) sh.top[r] = best;
    last = best;
    __syncthreads();
    if (!best) break;
  }
}

__global__ void __launch_bounds__(kThreads, 8) k_token_logprobs(Args a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = 1 << a.split, rank = (int)(blockIdx.x & (split - 1));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x >> a.split;
  Slice s;
  s.row = a.logits + row * a.row_stride;
  s.vocab = a.vocab;
  s.lead = (int)((reinterpret_cast<uintptr_t>(s.row) >> 2) & 3);
  const int all = (a.vocab + s.lead + 3) / 4;
  s.c0 = min(rank * a.chunks, all);
  s.n = min(a.chunks, all - s.c0);
  const int k = a.top_k;

  // the tokens (the first CTA's first warp), on their way meanwhile
  int id[QD_MAX_TREE / 32];
#pragma unroll
  for (int j = 0; j < QD_MAX_TREE / 32; ++j) {
    const int t = tid + 32 * j;
    id[j] = rank == 0 && warp == 0 && t < a.n_tokens ? a.tokens[row * a.n_tokens + t] : -1;
  }
  if (tid < QD_MAX_TOP) sh.top[tid] = 0;
  if (tid == 0) {
    sh.count = sh.reached = 0;
    sh.owner = kThreads;
  }
  if (split > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // this CTA runs

  // ---- the stream: thread t has chunks t, t + 256, ...
  Running run{-INFINITY, 0.f, 0.f};
  {
    // chunks [lo, hi) lie inside the row; the row's first and last may not
    const int lo = s.c0 == 0 && s.lead ? 1 : 0;
    const int hi = min(s.n, (a.vocab + s.lead) / 4 - s.c0);
    const float4* src = reinterpret_cast<const float4*>(s.row + s.index(0));
    constexpr int kStep = kBatch * kThreads;
    int c = tid;
    float4 x[kBatch], y[kBatch];
    auto load = [&](float4 (&to)[kBatch]) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) to[j] = __ldcg(src + c + j * kThreads);
    };
    auto load_edge = [&](float4 (&to)[kBatch]) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int at = c + j * kThreads;
        to[j] = at >= lo && at < hi ? __ldcg(src + at)
                : at < s.n          ? s.read(at)
                                    : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      }
    };
    if (lo && s.n > 0) {  // the row begins inside a chunk: its first batch is an edge
      load_edge(x);
      run.add(x);
      c += kStep;
    }
    if (c + kStep - kThreads < hi) {
      load(x);
      c += kStep;
      for (; c + kStep - kThreads < hi; c += kStep) {
        load(y);
        run.add(x);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) x[j] = y[j];
      }
      if (c < s.n) load_edge(y);
      run.add(x);
      if (c < s.n) run.add(y);
    } else if (c < s.n) {
      load_edge(x);
      run.add(x);
    }
  }

  float xt[QD_MAX_TREE / 32];
#pragma unroll
  for (int j = 0; j < QD_MAX_TREE / 32; ++j) xt[j] = id[j] >= 0 && id[j] < a.vocab ? __ldcg(s.row + id[j]) : -INFINITY;

  // ---- 1. the largest values
  const float tm = run.m;
  const float sorted = k > 1 ? warp_sort(tm, lane) : warp_max(tm);
  sh.wmax[warp][lane] = sorted;
  __syncthreads();
  const float m = warp_max(sh.wmax[lane & (kWarps - 1)][0]);
  if (tm == m) atomicMin(&sh.owner, tid);  // one thread that holds a largest value
  if (warp == 0) {
    float v = sorted;
    if (k > 1)
#pragma unroll
      for (int w = 1; w < kWarps; ++w) v = warp_merge(v, sh.wmax[w][31 - lane], lane);
    if (lane == max(k - 1, 0)) sh.bound = k > 1 ? v : m;
  }
  __syncthreads();
  const float bound = sh.bound;
  const bool list = k > 0 && bound > -INFINITY;
  const int owner = m > -INFINITY ? sh.owner : -1;
  if ((list && tm >= bound) || tid == owner) sh.reach[atomicAdd(&sh.reached, 1)] = (uint8_t)tid;
  {  // the slice's sums, in units of its largest value; the owner's follow
    const float d = max_nan(fmaxf(tm, kLowest) - fmaxf(m, kLowest), -1e4f), f = ex2(d * 1.4426950408889634f);
    const float r = warp_sum(tid == owner ? 0.f : f * run.r);
    const float h = warp_sum(tid == owner ? 0.f : f * fmaf(d, run.r, run.h));
    if (lane == 0) sh.warp[warp] = Part{m, r, h};
    if (tid == 0) sh.own = make_float2(0.f, 0.f);
  }
  __syncthreads();
  for (int x = warp; x < sh.reached; x += kWarps) {  // a warp reads a thread's values again
    const int t = sh.reach[x];
    Running again{m, 0.f, 0.f};
    bool skip = t == owner;
    for (int i = t; i < s.n; i += 32 * kThreads) {
      const int c = i + lane * kThreads;
      const float4 v = c < s.n ? s.read(c) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      const float e[4] = {v.x, v.y, v.z, v.w};
      const float top = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
      if (list && top >= bound) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e[j] >= bound) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kList) sh.list[at] = order_key(e[j], s.index(c) + j);
          }
      }
      if (t == owner) {
        const unsigned holds = __ballot_sync(0xffffffffu, top == m);
        bool out = skip && holds && lane == __ffs(holds) - 1;
        skip = skip && !holds;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool here = out && e[j] == m;
          again.add(here ? -INFINITY : e[j], m);
          out = out && !here;
        }
      }
    }
    if (t == owner) {
      const float r = warp_sum(again.r), h = warp_sum(again.h);
      if (lane == 0) sh.own = make_float2(r, h);
    }
  }
  __syncthreads();
  if (k > 0) {
    const int n = sh.count;
    if (list && n <= kList) {
      rank_list(sh.list, n, k, sh.top);
      if (n > 32) __syncthreads();  // otherwise the first warp has ranked them all
    } else if (s.n > 0) {
      select_slow(s, bound, k, sh);
    }
  }

  // ---- 2. the first warp of the cluster's first CTA joins the slices
  Part p{m, 0.f, 0.f};
  if (warp == 0) {
    __syncwarp();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      p.r += sh.warp[w].r;
      p.h += sh.warp[w].h;
    }
    p.r += sh.own.x;
    p.h += sh.own.y;
  }
  if (split > 1) {
    asm volatile("barrier.cluster.wait;" ::: "memory");  // the first CTA runs
    if (warp == 0) {
      if (lane == 0) *cluster.map_shared_rank(&sh.parts[rank], 0) = p;
      if (lane < k) *cluster.map_shared_rank(&sh.tops[rank][lane], 0) = sh.top[lane];
    }
    cluster.sync();
  }
  if (rank != 0 || warp != 0) return;
  u64 key = lane < k ? sh.top[lane] : 0;
  if (split > 1) {
    Part q{-INFINITY, 0.f, 0.f};
    if (lane < split) q = sh.parts[lane];
    const float top = warp_max(q.m);
    const int out = __ffs(__ballot_sync(0xffffffffu, q.m == top)) - 1;  // the slice that left a largest value out
    float pr, ph;
    if (q.m == -INFINITY) {  // nothing but -INFINITY (r = 0) or NaN
      pr = q.r;
      ph = 0.f;
    } else if (lane == out) {
      pr = q.r;
      ph = q.h;
    } else {
      const float d = max_nan(q.m - top, -1e4f), f = ex2(d * 1.4426950408889634f);
      pr = f * (1.f + q.r);
      ph = f * fmaf(d, 1.f + q.r, q.h);
    }
    p = Part{top, warp_sum(pr), warp_sum(ph)};
    for (int c = 1; c < split; ++c) key = warp_merge(key, 31 - lane < k ? sh.tops[c][31 - lane] : 0ull, lane);
  }
  // without a finite largest value x - m has no value for any token
  const float lse = fabsf(p.m) < INFINITY ? log1pf(p.r) : NAN;
  if (lane == 0 && a.entropy) a.entropy[row] = lse - p.h / (1.f + p.r);
#pragma unroll
  for (int j = 0; j < QD_MAX_TREE / 32; ++j) {
    const int t = lane + 32 * j;
    if (t < a.n_tokens)
      a.logprob[row * a.n_tokens + t] = id[j] >= 0 && id[j] < a.vocab ? (xt[j] - p.m) - lse : -INFINITY;
  }
  if (lane < k) {
    a.top_idx[row * k + lane] = (int32_t)argmax_key_index(key);
    a.top_logprob[row * k + lane] = (key_value(key) - p.m) - lse;
  }
}

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_token_logprobs(const float* logits, int64_t row_stride, int64_t vocab, int rows, const int32_t* tokens,
                            int n_tokens, float* logprob, float* entropy, int top_k, int32_t* top_idx,
                            float* top_logprob, qd_stream_t stream) {
  if (!logits) return QD_ERR_INVALID_ARG;
  if (vocab < 1 || vocab > QD_MAX_VOCAB || rows < 1 || rows > QD_MAX_GEMM_TOKENS || n_tokens < 0 ||
      n_tokens > QD_MAX_TREE || top_k < 0 || top_k > QD_MAX_TOP || top_k > vocab)
    return QD_ERR_SHAPE;
  if (rows > 1 && row_stride < vocab) return QD_ERR_SHAPE;
  if (n_tokens && (!tokens || !logprob)) return QD_ERR_INVALID_ARG;
  if (top_k && (!top_idx || !top_logprob)) return QD_ERR_INVALID_ARG;
  if (!n_tokens && !top_k && !entropy) return QD_ERR_INVALID_ARG;  // nothing asked for
  if (!aligned16(logits) || (n_tokens && (!aligned4(tokens) || !aligned4(logprob))) || !aligned4(entropy) ||
      (top_k && (!aligned4(top_idx) || !aligned4(top_logprob))))
    return QD_ERR_ALIGN;
  // CTAs to a row: one, and more while SMs lack the four CTAs that fit and a thread would still
  // have two batches
  const int64_t chunks = (vocab + 3 + 3) / 4;  // of a row, wherever it starts
  int log_split = 0;
  while ((1 << log_split) < kMaxSplit && ((int64_t)rows << log_split) < 4 * attn_sm_count() &&
         chunks >= ((int64_t)4 * kBatch * kThreads << log_split))
    ++log_split;
  const int split = 1 << log_split;
  Args a;
  a.logits = logits;
  a.row_stride = row_stride;
  a.vocab = (int)vocab;
  a.tokens = tokens;
  a.n_tokens = n_tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_k = top_k;
  a.top_idx = top_idx;
  a.top_logprob = top_logprob;
  a.chunks = (int)((chunks + split - 1) / split);
  a.split = log_split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * split));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_token_logprobs, a) == cudaSuccess ? QD_OK : QD_ERR_CUDA;
}

}  // extern "C"
