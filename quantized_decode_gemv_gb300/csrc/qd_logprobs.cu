// Log probabilities of given tokens, entropy and the top alternatives of rows of logits.
// With m = max x and r = sum over all but one of the largest of e^(x - m):
//   log p_t = (x_t - m) - log1p(r)
//   H       = log1p(r) - sum e^(x - m) (x - m) / (1 + r)
// Both terms of H are positive and r leaves the largest out, so neither loses digits when one
// token holds nearly all of the probability.
#include "qd_internal.cuh"

namespace qd {
namespace {

constexpr int kThreads = 1024;

struct Best {
  float v;
  int i;
};
// Larger value first, then the lower index; NaN after everything (v >= w is false for it).
__device__ __forceinline__ bool before(Best a, Best b) {
  const bool an = a.v != a.v, bn = b.v != b.v;
  if (an || bn) return an == bn ? a.i < b.i : bn;
  return a.v > b.v || (a.v == b.v && a.i < b.i);
}

__device__ __forceinline__ Best block_best(Best x, Best* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Best y{__shfl_xor_sync(0xffffffffu, x.v, o), __shfl_xor_sync(0xffffffffu, x.i, o)};
    if (before(y, x)) x = y;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Best y{__shfl_xor_sync(0xffffffffu, x.v, o), __shfl_xor_sync(0xffffffffu, x.i, o)};
    if (before(y, x)) x = y;
  }
  return x;
}

__global__ void __launch_bounds__(kThreads) k_token_logprobs(const float* __restrict__ logits, int64_t row_stride,
                                                             int vocab, const int32_t* __restrict__ tokens,
                                                             int n_tokens, float* __restrict__ logprob,
                                                             float* __restrict__ entropy, int top_k,
                                                             int32_t* __restrict__ top_idx,
                                                             float* __restrict__ top_logprob) {
  __shared__ Best red[32];
  __shared__ float2 sums[32];
  const int64_t row = blockIdx.x;
  const float* x = logits + row * row_stride;
  Best b{NAN, 0x7FFFFFFF};
  for (int i = threadIdx.x; i < vocab; i += kThreads) {
    const Best y{x[i], i};
    if (before(y, b)) b = y;
  }
  b = block_best(b, red);
  const float m = b.v;
  const int first = b.i;
  float r = 0.f, h = 0.f;
  for (int i = threadIdx.x; i < vocab; i += kThreads) {
    const float d = x[i] - m;
    const float e = expf(d);
    if (i != first) {
      r += e;
      h += d == -INFINITY ? 0.f : e * d;
    }
  }
  r = warp_sum(r);
  h = warp_sum(h);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_float2(r, h);
  __syncthreads();
  const float2 s = sums[threadIdx.x & 31];
  r = warp_sum(s.x);
  h = warp_sum(s.y);
  // without a finite maximum x - m has no value for any token
  const float lse = fabsf(m) < INFINITY ? log1pf(r) : NAN;
  if (threadIdx.x == 0 && entropy) entropy[row] = lse - h / (1.f + r);
  for (int t = threadIdx.x; t < n_tokens; t += kThreads) {
    const int id = tokens[row * n_tokens + t];
    logprob[row * n_tokens + t] = id >= 0 && id < vocab ? (x[id] - m) - lse : -INFINITY;
  }
  Best last = b;
  for (int k = 0; k < top_k; ++k) {
    if (k) {
      b = Best{NAN, 0x7FFFFFFF};
      for (int i = threadIdx.x; i < vocab; i += kThreads) {
        const Best y{x[i], i};
        if (before(last, y) && before(y, b)) b = y;
      }
      last = b = block_best(b, red);
    }
    if (threadIdx.x == 0) {
      top_idx[row * top_k + k] = b.i;
      top_logprob[row * top_k + k] = (b.v - m) - lse;
    }
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
  if (!aligned16(logits)) return QD_ERR_ALIGN;
  k_token_logprobs<<<rows, kThreads, 0, (cudaStream_t)stream>>>(logits, row_stride, (int)vocab, tokens, n_tokens,
                                                                logprob, entropy, top_k, top_idx, top_logprob);
  return launch_status();
}

}  // extern "C"
