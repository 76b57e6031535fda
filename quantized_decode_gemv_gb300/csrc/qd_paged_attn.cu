// Causal attention of packed rows over the pages of an 8-bit cache:
//   o = sum_j softmax_j(scale q . k_j) v_j,  k_j = code * scale of its block, over the positions
// j = 0 .. p of a row at position p (the last `window` of them with a window).
#include <algorithm>

#include "qd_paged.cuh"

namespace qd {
namespace {

using paged::Cache;

struct AttnArgs {
  Cache c;
  const float* q;
  int64_t q_stride;
  float* out;
  int n_heads, n_tokens, n_seqs, group;
  const int32_t *row_start, *pos;
  float scale;
  int window;
};

template <int FMT>
__device__ __forceinline__ float value_of(uint8_t w) {
  if constexpr (FMT == QD_KV_I8) return (float)(int8_t)w;
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

// A warp a row and head, a running maximum and sum, one position at a time.
template <int HD, int FMT>
__global__ void k_paged_attn(AttnArgs a) {
  constexpr int kPer = HD / 32;
  const int row = blockIdx.x, kvh = blockIdx.y, h = kvh * a.group + threadIdx.y, lane = threadIdx.x;
  int before = 0;
  for (int b = lane; b < a.n_seqs; b += 32) before += a.row_start[b] <= row;
  before = __reduce_add_sync(0xffffffffu, before);
  if (!before || row >= a.row_start[before]) return;
  const int seq = before - 1;
  int row0;
  const int t = paged::rows_of(a.row_start, seq, a.n_tokens, row0);
  const int p0 = a.pos[seq];
  float o[kPer] = {}, q[kPer], m = -INFINITY, l = 0.f;
  if (p0 >= 0 && (int64_t)p0 + t <= a.c.capacity) {
    const int p = p0 + row - row0;
    for (int i = 0; i < kPer; ++i) q[i] = a.q[row * a.q_stride + (int64_t)h * HD + lane * kPer + i] * a.scale;
    for (int j = a.window > 0 ? max(p - a.window + 1, 0) : 0; j <= p; ++j) {
      int in_page;
      const int page = paged::page_of(a.c, seq, j / QD_KV_BLOCK, in_page);
      const int64_t at = page < 0 ? 0 : paged::block_index(a.c, page, kvh, in_page);
      const float nan = __uint_as_float(0x7FC00000u);
      const float ks = page < 0 ? nan : a.c.ks[at], vs = page < 0 ? nan : a.c.vs[at];
      const int64_t e = at * (16 * HD) + j % QD_KV_BLOCK * HD + lane * kPer;
      float s = 0.f;
      for (int i = 0; i < kPer; ++i) s += q[i] * value_of<FMT>(a.c.k[e + i]);
      s = warp_sum(s) * ks;
      const float mn = s > m || isnan(s) ? s : m, keep = expf(m - mn), w = expf(s - mn);
      l = l * keep + w;
      for (int i = 0; i < kPer; ++i) o[i] = o[i] * keep + w * vs * value_of<FMT>(a.c.v[e + i]);
      m = mn;
    }
    for (int i = 0; i < kPer; ++i) o[i] /= l;
  }
  for (int i = 0; i < kPer; ++i) a.out[((int64_t)row * a.n_heads + h) * HD + lane * kPer + i] = o[i];
}

inline bool attn_shape_ok(const qd_paged_kv* kv, int n_heads, int n_tokens, int n_seqs) {
  return paged::cache_status(kv, n_seqs) == QD_OK && n_heads >= 1 && n_heads % kv->n_kv_heads == 0 &&
         n_heads / kv->n_kv_heads <= 16 && n_tokens >= 1 && n_tokens <= QD_MAX_GEMM_TOKENS;
}

}  // namespace
}  // namespace qd

using namespace qd;

extern "C" {

size_t qd_paged_attn_workspace(const qd_paged_kv* kv, int n_heads, int n_tokens, int n_seqs) {
  return attn_shape_ok(kv, n_heads, n_tokens, n_seqs) ? 16 : 0;
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
  AttnArgs a = {paged::cache_of(kv), q, q_stride, out, n_heads, n_tokens, n_seqs, n_heads / kv->n_kv_heads,
                row_start, pos, scale, window};
  const dim3 grid((unsigned)n_tokens, (unsigned)kv->n_kv_heads), block(32, (unsigned)a.group);
  cudaStream_t st = (cudaStream_t)stream;
  if (kv->head_dim == 64) {
    if (kv->fmt == QD_KV_I8) k_paged_attn<64, QD_KV_I8><<<grid, block, 0, st>>>(a);
    else k_paged_attn<64, QD_KV_E4M3><<<grid, block, 0, st>>>(a);
  } else {
    if (kv->fmt == QD_KV_I8) k_paged_attn<128, QD_KV_I8><<<grid, block, 0, st>>>(a);
    else k_paged_attn<128, QD_KV_E4M3><<<grid, block, 0, st>>>(a);
  }
  return launch_status();
}

}  // extern "C"
