// Attention of a tree of drafted tokens over the cache: node i of sequence b sees the pos[b]
// cached positions and the draft slots j with bit j of its mask set,
//   o = sum_p softmax_p(q . k_p / sqrt(head_dim)) v_p.
#include "qd_internal.cuh"

namespace qd {
namespace {

constexpr int kHd = 64;

template <typename KV>
__device__ __forceinline__ float2 load2(const KV* p);
template <>
__device__ __forceinline__ float2 load2<float>(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}
template <>
__device__ __forceinline__ float2 load2<__half>(const __half* p) {
  return __half22float2(*reinterpret_cast<const __half2*>(p));
}

// One warp per (head, node, sequence); a lane holds dimensions 2 lane, 2 lane + 1.
template <typename KV>
__global__ void __launch_bounds__(32) k_tree_attn(const float* __restrict__ q, int64_t q_batch_stride,
                                                  const KV* __restrict__ kc, const KV* __restrict__ vc,
                                                  const KV* __restrict__ kd, const KV* __restrict__ vd,
                                                  float* __restrict__ out, int n_kv, const int32_t* __restrict__ pos,
                                                  const uint64_t* __restrict__ mask,
                                                  const int32_t* __restrict__ n_valid, int n_nodes, int max_ctx) {
  const int h = blockIdx.x, node = blockIdx.y, b = blockIdx.z, lane = threadIdx.x;
  const int n_heads = gridDim.x, kvh = h / (n_heads / n_kv);
  const int cnt = n_valid ? min(max(n_valid[b], 0), n_nodes) : n_nodes;
  if (node >= cnt) return;
  const int p0 = pos[b];
  float2* dst = reinterpret_cast<float2*>(out + (((int64_t)b * n_nodes + node) * n_heads + h) * kHd) + lane;
  if (p0 < 0 || p0 > max_ctx) {
    *dst = make_float2(0.f, 0.f);
    return;
  }
  const float2 qv =
      load2(q + (int64_t)b * q_batch_stride + ((int64_t)node * n_heads + h) * kHd + 2 * lane);
  const int64_t head = (int64_t)b * n_kv + kvh;
  const uint64_t sees = mask[(int64_t)b * n_nodes + node];
  float m = -INFINITY, l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  auto step = [&](const KV* k, const KV* v) {
    const float2 kv = load2(k + 2 * lane);
    const float s = warp_sum(qv.x * kv.x + qv.y * kv.y) * (1.4426950408889634f * 0.125f);
    const float mn = fmaxf(m, s);
    const float corr = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
    const float2 vv = load2(v + 2 * lane);
    l = l * corr + w;
    o.x = o.x * corr + w * vv.x;
    o.y = o.y * corr + w * vv.y;
    m = mn;
  };
  for (int p = 0; p < p0; ++p) {
    const int64_t at = (head * max_ctx + p) * kHd;
    step(kc + at, vc + at);
  }
  for (int j = 0; j < cnt; ++j)
    if (sees >> j & 1) {
      const int64_t at = (head * n_nodes + j) * kHd;
      step(kd + at, vd + at);
    }
  *dst = l == 0.f ? make_float2(0.f, 0.f) : make_float2(o.x / l, o.y / l);
}

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

size_t qd_tree_attn_workspace(int n_heads, int n_kv_heads, int head_dim, int n_nodes, int max_ctx, int batch) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > 8 || head_dim != kHd ||
      n_nodes < 1 || n_nodes > QD_MAX_TREE || max_ctx < 1 || batch < 1 || batch > QD_MAX_BATCH)
    return 0;
  return 256;
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
  if (!need || n_heads > 65535) return QD_ERR_SHAPE;
  if (batch > 1 && q_batch_stride < (int64_t)n_nodes * n_heads * head_dim) return QD_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_draft) || !aligned16(v_draft) ||
      !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(mask) & 7) ||
      ((reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(n_valid)) & 3))
    return QD_ERR_ALIGN;
  if (batch > 1 && q_batch_stride % 4) return QD_ERR_ALIGN;
  if (workspace_bytes < need) return QD_ERR_NOMEM;
  const dim3 grid((unsigned)n_heads, (unsigned)n_nodes, (unsigned)batch);
  cudaStream_t st = (cudaStream_t)stream;
  if (kv_f16)
    k_tree_attn<__half><<<grid, 32, 0, st>>>(q, q_batch_stride, static_cast<const __half*>(k_cache),
                                             static_cast<const __half*>(v_cache), static_cast<const __half*>(k_draft),
                                             static_cast<const __half*>(v_draft), out, n_kv_heads, pos, mask, n_valid,
                                             n_nodes, max_ctx);
  else
    k_tree_attn<float><<<grid, 32, 0, st>>>(q, q_batch_stride, static_cast<const float*>(k_cache),
                                            static_cast<const float*>(v_cache), static_cast<const float*>(k_draft),
                                            static_cast<const float*>(v_draft), out, n_kv_heads, pos, mask, n_valid,
                                            n_nodes, max_ctx);
  return launch_status();
}

}  // extern "C"
