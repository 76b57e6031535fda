// Verification of a tree of drafted tokens: the host-side plan of a tree (ancestor masks and
// depths), the rotation and storage of its queries, keys and values, and the walk that accepts
// a path and copies its rows into the cache.  The attention between the two is
// qd_tree_attn.cu, the scores of the drafted tokens qd_logprobs.cu.
#include <algorithm>

#include "qd_internal.cuh"

namespace qd {
namespace {

// ------------------------------------------------------------------ append
// q' = R(pos + depth) q and k' = R(pos + depth) k, pair by pair (x0 c - x1 s, x0 s + x1 c),
// v copied; k' and v rounded once to the cache's type.  A thread takes 8 elements of a head
// (4 pairs): two 16-byte loads of values, two of (cos, sin).
// A pass is one read and one write of each row, so the launch bounds a small tree and HBM a
// large one.
__device__ __forceinline__ void store4(float* p, float4 a) { *reinterpret_cast<float4*>(p) = a; }
__device__ __forceinline__ void store4(__half* p, float4 a) {
  __half2 h[2] = {__floats2half2_rn(a.x, a.y), __floats2half2_rn(a.z, a.w)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
}

template <typename KV>
__global__ void __launch_bounds__(256) k_tree_append(
    const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v, int64_t batch_stride,
    int64_t node_stride, float* __restrict__ q_out, KV* __restrict__ k_draft, KV* __restrict__ v_draft, int n_heads,
    int n_kv, int hd, const int32_t* __restrict__ pos, const int32_t* __restrict__ depth,
    const int32_t* __restrict__ n_valid, int n_nodes, int pairing, const float* __restrict__ cs, int max_ctx) {
  const int node = blockIdx.y, b = blockIdx.z;
  const int per_head = hd / 8;
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= (n_heads + 2 * n_kv) * per_head) return;
  if (n_valid && node >= n_valid[b]) return;
  const int p0 = pos[b], dp = depth[(int64_t)b * n_nodes + node];
  if (p0 < 0 || p0 >= max_ctx || dp < 0 || dp >= max_ctx - p0) return;
  const int h = u / per_head, i = u % per_head;
  const int64_t row = (int64_t)b * batch_stride + (int64_t)node * node_stride;
  const int half = hd / 2;
  if (h >= n_heads + n_kv) {
    const int hv = h - n_heads - n_kv;
    const float4* src = reinterpret_cast<const float4*>(v + row + (int64_t)hv * hd + 8 * i);
    KV* dst = v_draft + (((int64_t)b * n_kv + hv) * n_nodes + node) * hd + 8 * i;
    store4(dst, __ldcg(src));
    store4(dst + 4, __ldcg(src + 1));
    return;
  }
  const bool isq = h < n_heads;
  const float* src = isq ? q + row + (int64_t)h * hd : k + row + (int64_t)(h - n_heads) * hd;
  const float4* t = reinterpret_cast<const float4*>(cs + ((int64_t)(p0 + dp) * half + 4 * i) * 2);
  const float4 t0 = __ldg(t), t1 = __ldg(t + 1);  // (c, s) of pairs 4i..4i+3
  float4 a, o;                                    // the pairs' first and second elements
  int da, dob;
  if (pairing == QD_ROPE_HALF) {
    da = 4 * i;
    dob = half + 4 * i;
    const float4 x0 = __ldcg(reinterpret_cast<const float4*>(src + da));
    const float4 x1 = __ldcg(reinterpret_cast<const float4*>(src + dob));
    a = make_float4(x0.x * t0.x - x1.x * t0.y, x0.y * t0.z - x1.y * t0.w, x0.z * t1.x - x1.z * t1.y,
                    x0.w * t1.z - x1.w * t1.w);
    o = make_float4(x0.x * t0.y + x1.x * t0.x, x0.y * t0.w + x1.y * t0.z, x0.z * t1.y + x1.z * t1.x,
                    x0.w * t1.w + x1.w * t1.z);
  } else {
    da = 8 * i;
    dob = 8 * i + 4;
    const float4 x0 = __ldcg(reinterpret_cast<const float4*>(src + da));
    const float4 x1 = __ldcg(reinterpret_cast<const float4*>(src + dob));
    a = make_float4(x0.x * t0.x - x0.y * t0.y, x0.x * t0.y + x0.y * t0.x, x0.z * t0.z - x0.w * t0.w,
                    x0.z * t0.w + x0.w * t0.z);
    o = make_float4(x1.x * t1.x - x1.y * t1.y, x1.x * t1.y + x1.y * t1.x, x1.z * t1.z - x1.w * t1.w,
                    x1.z * t1.w + x1.w * t1.z);
  }
  if (isq) {
    float* dst = q_out + (((int64_t)b * n_nodes + node) * n_heads + h) * hd;
    store4(dst + da, a);
    store4(dst + dob, o);
  } else {
    KV* dst = k_draft + (((int64_t)b * n_kv + (h - n_heads)) * n_nodes + node) * hd;
    store4(dst + da, a);
    store4(dst + dob, o);
  }
}

// ------------------------------------------------------------------ commit
// The walk: from node 0, the next node is the first child (smallest index above the node's
// own) whose token is the one chosen after the node.  A warp holds the tree, two nodes to a
// lane, and finds each child with two ballots; every CTA walks for itself, which costs less
// than a second launch.  Then the accepted rows go from the draft buffers to positions
// pos + i of every layer's cache, 16 bytes a thread.
constexpr int kCommitThreads = 256;

__global__ void __launch_bounds__(kCommitThreads) k_tree_commit(
    const int32_t* __restrict__ tokens, const int32_t* __restrict__ parent, const int32_t* __restrict__ chosen,
    int64_t chosen_stride, const int32_t* __restrict__ n_valid, int n_nodes, const uint4* __restrict__ k_draft,
    const uint4* __restrict__ v_draft, uint4* __restrict__ k_cache, uint4* __restrict__ v_cache, int layers,
    int64_t layer_chunks, int n_kv, int row_chunks, const int32_t* __restrict__ pos, int max_ctx, int batch,
    int32_t* __restrict__ path, int32_t* __restrict__ n_accept, int32_t* __restrict__ next_token,
    int32_t* __restrict__ pos_out) {
  __shared__ int s_path[QD_MAX_TREE];
  __shared__ int s_len;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int p0 = pos[b];
  if (threadIdx.x < 32) {
    const int cnt = n_valid ? min(max(n_valid[b], 0), n_nodes) : n_nodes;
    const int most = p0 < 0 || p0 > max_ctx ? 0 : min(cnt, max_ctx - p0);  // rows the cache has room for
    int tok[2], par[2], cho[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = lane + 32 * j;
      const bool in = c < cnt;
      const int64_t at = (int64_t)b * n_nodes + c;
      tok[j] = in ? tokens[at] : 0;
      par[j] = in && c > 0 ? parent[at] : -1;
      cho[j] = in ? chosen[at * chosen_stride] : -1;
    }
    int len = 0, cur = 0, want = -1;
    while (len < most) {  // cur grows with every step, so there are at most QD_MAX_TREE
      if (lane == 0) s_path[len] = cur;
      ++len;
      const int w0 = __shfl_sync(0xffffffffu, cho[0], cur & 31), w1 = __shfl_sync(0xffffffffu, cho[1], cur & 31);
      want = cur < 32 ? w0 : w1;
      const unsigned m0 = __ballot_sync(0xffffffffu, lane < cnt && par[0] == cur && lane > cur && tok[0] == want);
      const unsigned m1 =
          __ballot_sync(0xffffffffu, lane + 32 < cnt && par[1] == cur && lane + 32 > cur && tok[1] == want);
      if (!(m0 | m1)) break;
      cur = m0 ? __ffs(m0) - 1 : __ffs(m1) + 31;
    }
    if (lane == 0) s_len = len;
    if (blockIdx.x == 0) {
      __syncwarp();
      for (int c = lane; c < n_nodes; c += 32) path[(int64_t)b * n_nodes + c] = c < len ? s_path[c] : -1;
      if (lane == 0) {
        n_accept[b] = len;
        next_token[b] = want;
        pos_out[b] = p0 + len;
      }
    }
  }
  __syncthreads();
  const int per = s_len * row_chunks;  // 16-byte chunks of one (layer, kv head)
  if (!per) return;
  for (int pair = blockIdx.x; pair < layers * n_kv; pair += gridDim.x) {
    const int l = pair / n_kv, h = pair % n_kv;
    const int64_t src = (((int64_t)l * batch + b) * n_kv + h) * n_nodes * row_chunks;
    const int64_t dst = (int64_t)l * layer_chunks + (((int64_t)b * n_kv + h) * max_ctx + p0) * row_chunks;
    for (int t = threadIdx.x; t < 2 * per; t += kCommitThreads) {
      const bool isv = t >= per;
      const int e = isv ? t - per : t;
      const int r = e / row_chunks, c = e % row_chunks;
      const int64_t s = src + (int64_t)s_path[r] * row_chunks + c;
      (isv ? v_cache : k_cache)[dst + e] = __ldcg((isv ? v_draft : k_draft) + s);
    }
  }
}

inline bool kv_shape_ok(int head_dim) { return head_dim >= 8 && head_dim <= 1024 && head_dim % 8 == 0; }

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_tree_plan(const int32_t* parent_host, int n_nodes, uint64_t* mask_host, int32_t* depth_host) {
  if (n_nodes < 1 || n_nodes > QD_MAX_TREE) return QD_ERR_SHAPE;
  if (!parent_host || !mask_host || !depth_host) return QD_ERR_INVALID_ARG;
  for (int i = 1; i < n_nodes; ++i)
    if (parent_host[i] < 0 || parent_host[i] >= i) return QD_ERR_INVALID_ARG;
  mask_host[0] = 1;
  depth_host[0] = 0;
  for (int i = 1; i < n_nodes; ++i) {
    mask_host[i] = mask_host[parent_host[i]] | (uint64_t(1) << i);
    depth_host[i] = depth_host[parent_host[i]] + 1;
  }
  return QD_OK;
}

qd_status qd_tree_append(const float* q, const float* k, const float* v, int64_t batch_stride, int64_t node_stride,
                         float* q_out, void* k_draft, void* v_draft, int kv_f16, int n_heads, int n_kv_heads,
                         int head_dim, const int32_t* pos, const int32_t* depth, const int32_t* n_valid, int n_nodes,
                         qd_rope_pairing pairing, const float* cos_sin, int max_ctx, int batch, qd_stream_t stream) {
  if (!q || !k || !v || !q_out || !k_draft || !v_draft || !pos || !depth || !cos_sin) return QD_ERR_INVALID_ARG;
  if (kv_f16 != 0 && kv_f16 != 1) return QD_ERR_INVALID_ARG;
  if (pairing != QD_ROPE_ADJACENT && pairing != QD_ROPE_HALF) return QD_ERR_UNSUPPORTED;
  if (n_heads < 1 || n_heads > 65536 || n_kv_heads < 1 || n_kv_heads > 65536 || !kv_shape_ok(head_dim) ||
      max_ctx < 1 || batch < 1 || batch > QD_MAX_BATCH || n_nodes < 1 || n_nodes > QD_MAX_TREE)
    return QD_ERR_SHAPE;
  const int64_t widest = (int64_t)std::max(n_heads, n_kv_heads) * head_dim;
  if ((n_nodes > 1 && node_stride < widest) || (batch > 1 && batch_stride < (n_nodes - 1) * node_stride + widest))
    return QD_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_draft) ||
      !aligned16(v_draft) || !aligned16(cos_sin) || !aligned4(pos) || !aligned4(depth) || !aligned4(n_valid))
    return QD_ERR_ALIGN;
  if ((batch > 1 && batch_stride % 4) || (n_nodes > 1 && node_stride % 4)) return QD_ERR_ALIGN;
  const int units = (n_heads + 2 * n_kv_heads) * (head_dim / 8);
  const dim3 grid((unsigned)((units + 255) / 256), (unsigned)n_nodes, (unsigned)batch);
  cudaStream_t st = (cudaStream_t)stream;
  if (kv_f16)
    k_tree_append<__half><<<grid, 256, 0, st>>>(q, k, v, batch_stride, node_stride, q_out,
                                                static_cast<__half*>(k_draft), static_cast<__half*>(v_draft), n_heads,
                                                n_kv_heads, head_dim, pos, depth, n_valid, n_nodes, pairing, cos_sin,
                                                max_ctx);
  else
    k_tree_append<float><<<grid, 256, 0, st>>>(q, k, v, batch_stride, node_stride, q_out,
                                               static_cast<float*>(k_draft), static_cast<float*>(v_draft), n_heads,
                                               n_kv_heads, head_dim, pos, depth, n_valid, n_nodes, pairing, cos_sin,
                                               max_ctx);
  return launch_status();
}

qd_status qd_tree_commit(const int32_t* tokens, const int32_t* parent, const int32_t* chosen, int64_t chosen_stride,
                         const int32_t* n_valid, int n_nodes, const void* k_draft, const void* v_draft, void* k_cache,
                         void* v_cache, int kv_f16, int layers, int64_t cache_layer_stride, int n_kv_heads,
                         int head_dim, const int32_t* pos, int max_ctx, int batch, int32_t* path, int32_t* n_accept,
                         int32_t* next_token, int32_t* pos_out, qd_stream_t stream) {
  if (!tokens || !parent || !chosen || !k_draft || !v_draft || !k_cache || !v_cache || !pos || !path || !n_accept ||
      !next_token || !pos_out)
    return QD_ERR_INVALID_ARG;
  if ((kv_f16 != 0 && kv_f16 != 1) || chosen_stride < 1) return QD_ERR_INVALID_ARG;
  if (layers < 1 || layers > 65536 || n_kv_heads < 1 || n_kv_heads > 16384 || !kv_shape_ok(head_dim) || max_ctx < 1 ||
      batch < 1 || batch > QD_MAX_BATCH || n_nodes < 1 || n_nodes > QD_MAX_TREE)
    return QD_ERR_SHAPE;
  const int64_t cache = (int64_t)batch * n_kv_heads * max_ctx * head_dim;
  if (layers > 1 && cache_layer_stride < cache) return QD_ERR_SHAPE;
  const int esz = kv_f16 ? 2 : 4;
  if (!aligned16(k_draft) || !aligned16(v_draft) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(tokens) ||
      !aligned4(parent) || !aligned4(chosen) || !aligned4(n_valid) || !aligned4(pos) || !aligned4(path) ||
      !aligned4(n_accept) || !aligned4(next_token) || !aligned4(pos_out))
    return QD_ERR_ALIGN;
  if (layers > 1 && cache_layer_stride * esz % 16) return QD_ERR_ALIGN;
  if (pos == pos_out) return QD_ERR_INVALID_ARG;  // other CTAs still read pos
  const int pairs = layers * n_kv_heads;
  const int ctas = std::max(1, std::min(pairs, (8 * attn_sm_count() + batch - 1) / batch));
  k_tree_commit<<<dim3((unsigned)ctas, (unsigned)batch), kCommitThreads, 0, (cudaStream_t)stream>>>(
      tokens, parent, chosen, chosen_stride, n_valid, n_nodes, static_cast<const uint4*>(k_draft),
      static_cast<const uint4*>(v_draft), static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), layers,
      layers > 1 ? cache_layer_stride * esz / 16 : 0, n_kv_heads, head_dim * esz / 16, pos, max_ctx, batch, path,
      n_accept, next_token, pos_out);
  return launch_status();
}

}  // extern "C"
