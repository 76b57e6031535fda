// Log probabilities of given tokens, entropy and the top alternatives of rows of logits.
// With m = max x, and r and h the sums of e^(x - m) and e^(x - m) (x - m) over all values but
// one largest,
//   log p_t = (x_t - m) - log1p(r)
//   H       = log1p(r) - h / (1 + r)
// Both terms of H are positive and r leaves the largest out, so neither loses digits when one
// token holds nearly all of the probability.  Parts (m, r, h) join as
//   (1 + r_a) e^(m_a - m) and (h_a + (m_a - m) (1 + r_a)) e^(m_a - m).
//
// HBM bounds the call: 4 bytes and about ten instructions a value.  A row goes to a cluster of
// 1 to 8 CTAs; each copies its slice to shared memory once (16-byte asynchronous copies, every
// byte of the slice in flight at the same time) and takes all passes from there:
//  1. a running maximum per thread.  The k-th largest of the 256 threads' maxima (a bitonic sort
//     per warp and a merge tree) is at most the slice's k-th largest value;
//  2. the sums, and a list of the values at or above that bound: k of them and few more, as a
//     thread seldom holds two.  A list that overflows (many equal values) falls back to the
//     values above the bound and an ordered scan for those equal to it;
//  3. the list is ranked by counting, the slices' results are joined by the cluster's first CTA
//     through distributed shared memory.
// No atomic's order shows: the list is ranked by (value, index), sums have a fixed order.
#include <cooperative_groups.h>

#include <algorithm>

#include "qd_internal.cuh"
#include "qd_tc.cuh"

namespace qd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 256;           // values at or above the bound that are ranked at once
constexpr int kMaxSplit = 8;         // CTAs to a row
constexpr int kMaxChunks = 12800;    // 16-byte chunks of a slice in shared memory (200 KB)
constexpr int kGoodChunks = 3072;    // 48 KB: four CTAs to an SM
static_assert(kMaxSplit * QD_MAX_TOP <= kList, "the slices' lists are ranked like one");

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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
// The 32 largest of two falling lists, falling.
__device__ __forceinline__ float warp_merge(float a, const float* b, int lane) {
  float v = fmaxf(a, b[31 - lane]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = sort_step(v, o, false, lane);
  return v;
}

struct Part {
  float m, r, h;
};
struct Shared {
  float wmax[kWarps][32];
  Part warp[kWarps];
  Part part;             // of the slice
  u64 list[kList];
  u64 top[QD_MAX_TOP];   // the slice's largest, falling; 0: none
  int count, owner;
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
};

// The slice: chunk c of the row's 16-byte aligned span holds values 4 c - lead .. 4 c - lead + 3;
// this CTA has chunks [c0, c0 + n), the first `held` of them in shared memory.  What lies
// outside the row reads as -INFINITY.
struct Slice {
  const float* row;
  const float4* held_at;
  int vocab, lead, c0, n, held;
  __device__ __forceinline__ int index(int c) const { return 4 * (c0 + c) - lead; }
  __device__ __forceinline__ float at(int i) const { return i >= 0 && i < vocab ? __ldcg(row + i) : -INFINITY; }
  __device__ __forceinline__ bool inside(int c) const { return index(c) >= 0 && index(c) + 3 < vocab; }
  __device__ __forceinline__ float4 read(int c) const {
    const int i = index(c);
    if (inside(c)) return __ldcg(reinterpret_cast<const float4*>(row + i));
    return make_float4(at(i), at(i + 1), at(i + 2), at(i + 3));
  }
  __device__ __forceinline__ float4 get(int c) const { return c < held ? held_at[c] : read(c); }
  __device__ __forceinline__ float value(int e) const {  // value e of the slice
    if ((e >> 2) < held) return reinterpret_cast<const float*>(held_at)[e];
    return at(4 * c0 - lead + e);
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
    const float v = in ? s.value(e) : 0.f;
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
    const float4 x = s.get(c);
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
      const float4 x = s.get(c);
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

__global__ void __launch_bounds__(kThreads) k_token_logprobs(Args a) {
  extern __shared__ __align__(16) float4 held[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x / split;
  Slice s;
  s.row = a.logits + row * a.row_stride;
  s.held_at = held;
  s.vocab = a.vocab;
  s.lead = (int)((reinterpret_cast<uintptr_t>(s.row) >> 2) & 3);
  const int all = (a.vocab + s.lead + 3) / 4;
  s.c0 = min(rank * a.chunks, all);
  s.n = min(a.chunks, all - s.c0);
  s.held = min(s.n, kMaxChunks);

  for (int c = tid; c < s.held; c += kThreads) {
    if (s.inside(c))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(held + c)), "l"(s.row + s.index(c))
                   : "memory");
    else
      held[c] = s.read(c);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  // the tokens' own logits, on their way meanwhile
  float xt = -INFINITY;
  bool known = false;
  if (rank == 0 && tid < a.n_tokens) {
    const int id = a.tokens[row * a.n_tokens + tid];
    known = id >= 0 && id < a.vocab;
    if (known) xt = __ldcg(s.row + id);
  }
  if (tid < QD_MAX_TOP) sh.top[tid] = 0;
  if (tid == 0) {
    sh.count = 0;
    sh.owner = kThreads;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");  // a thread reads its own chunks alone until the barrier

  // ---- 1. maxima
  float tm = -INFINITY;
  for (int c = tid; c < s.n; c += kThreads) {
    const float4 x = s.get(c);
    tm = fmaxf(tm, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
  }
  const int k = a.top_k;
  float v = k > 1 ? warp_sort(tm, lane) : warp_max(tm);
  sh.wmax[warp][lane] = v;
  __syncthreads();
  float m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh.wmax[w][0]);
  if (tm == m) atomicMin(&sh.owner, tid);  // one thread that holds a largest value
  float bound = m;
  if (k > 1) {
#pragma unroll
    for (int w = kWarps / 2; w > 0; w >>= 1) {
      __syncthreads();
      if (warp < w) {
        v = warp_merge(v, sh.wmax[warp + w], lane);
        sh.wmax[warp][lane] = v;
      }
    }
    __syncthreads();
    bound = sh.wmax[0][k - 1];
  } else {
    __syncthreads();
  }

  // ---- 2. sums, and the values at or above the bound
  const float mu = fabsf(m) < INFINITY ? m : 0.f;
  bool skip = sh.owner == tid && m > -INFINITY;  // leaves one largest value out
  const bool list = k > 0 && bound > -INFINITY;
  float r = 0.f, h = 0.f;
  for (int c = tid; c < s.n; c += kThreads) {
    const float4 x = s.get(c);
    const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float d = max_nan(e[j] - mu, -1e4f);  // finite: 0 times it is 0
      const float p = ex2(d * 1.4426950408889634f);
      if (skip && e[j] == m) {
        skip = false;
      } else {
        r += p;
        h = fmaf(p, d, h);
      }
    }
    if (list && fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) >= bound) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e[j] >= bound) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kList) sh.list[at] = order_key(e[j], s.index(c) + j);
        }
    }
  }
  r = warp_sum(r);
  h = warp_sum(h);
  if (lane == 0) sh.warp[warp] = Part{m, r, h};
  __syncthreads();
  if (tid == 0) {
    Part p{m, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      p.r += sh.warp[w].r;
      p.h += sh.warp[w].h;
    }
    sh.part = p;
  }
  if (k > 0) {
    const int n = sh.count;
    if (list && n <= kList)
      rank_list(sh.list, n, k, sh.top);
    else if (s.n > 0)
      select_slow(s, bound, k, sh);
  }

  // ---- 3. the cluster's first CTA joins the slices
  cluster.sync();
  if (rank == 0) {
    Part p = sh.part;
    if (split > 1) {
      float top = p.m;
      for (int c = 1; c < split; ++c) top = fmaxf(top, cluster.map_shared_rank(&sh.part, c)->m);
      bool out = false;  // a largest value has been left out
      Part sum{top, 0.f, 0.f};
      for (int c = 0; c < split; ++c) {
        const Part q = *cluster.map_shared_rank(&sh.part, c);
        if (q.m == -INFINITY) {  // nothing but -INFINITY (r = 0) or NaN
          sum.r += q.r;
        } else if (q.m == top && !out) {
          out = true;
          sum.r += q.r;
          sum.h += q.h;
        } else {
          const float d = max_nan(q.m - top, -1e4f), f = ex2(d * 1.4426950408889634f);
          sum.r = fmaf(f, 1.f + q.r, sum.r);
          sum.h = fmaf(f, fmaf(d, 1.f + q.r, q.h), sum.h);
        }
      }
      p = sum;
      if (k > 0) {
        __syncthreads();
        for (int x = tid; x < split * k; x += kThreads) sh.list[x] = cluster.map_shared_rank(sh.top, x / k)[x % k];
        __syncthreads();
        rank_list(sh.list, split * k, k, sh.top);
      }
    }
    __syncthreads();
    // without a finite largest value x - m has no value for any token
    const float lse = fabsf(p.m) < INFINITY ? log1pf(p.r) : NAN;
    if (tid == 0 && a.entropy) a.entropy[row] = lse - p.h / (1.f + p.r);
    if (tid < a.n_tokens) a.logprob[row * a.n_tokens + tid] = known ? (xt - p.m) - lse : -INFINITY;
    if (tid < k) {
      const u64 key = sh.top[tid];
      a.top_idx[row * k + tid] = (int32_t)argmax_key_index(key);
      a.top_logprob[row * k + tid] = (key_value(key) - p.m) - lse;
    }
  }
  if (split > 1) cluster.sync();  // the other CTAs' shared memory has been read
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
  if (!aligned16(logits)) return QD_ERR_ALIGN;
  // CTAs to a row: slices of 48 KB or less, and more while there are SMs without a CTA and a
  // thread has two chunks
  const int64_t chunks = (vocab + 3 + 3) / 4;  // of a row, wherever it starts
  int split = 1;
  while (split < kMaxSplit &&
         (chunks > (int64_t)split * kGoodChunks ||
          ((int64_t)rows * split < attn_sm_count() && chunks >= (int64_t)split * 4 * kThreads)))
    split *= 2;
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
  const size_t smem = (size_t)std::min(a.chunks, kMaxChunks) * 16;
  if (smem > (48u << 10) - sizeof(Shared) &&
      cudaFuncSetAttribute(k_token_logprobs, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunks * 16) !=
          cudaSuccess)
    return QD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
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
