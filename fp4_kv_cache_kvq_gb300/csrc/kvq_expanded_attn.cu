// kvq_expanded_attn.cu -- causal attention of a chunk over dense keys and values
// whose key's position part is shared by all heads, and its C entry point.
//   y = softmax_scale log2 e (q[:d] . k + q[d:] . k_rope),
//   out = sum 2^(y - m) v / sum 2^(y - m)
#include "kvq_attn_rows.cuh"
#include "kvq_host.cuh"
#include "../../include/kvq_latent.h"

#include <cuda_bf16.h>

namespace kvq {
namespace {

struct ExpandedParams {
  const int32_t* lens;
  const int32_t* chunk_lens;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* kr;
  const uint16_t* v;
  void* out;
  int32_t* flag;
  int64_t k_ts, k_hs, kr_ts, v_ts, v_hs;
  int32_t batch, heads, d, rope, chunk, max_len, out_bf16, tiles;
  float scale_log2;
};

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

struct ExpandedSrc {
  const ExpandedParams& p;
  int b, h, r0;
  int64_t first;
  __device__ int64_t row(int r) const { return ((int64_t)b * p.chunk + r0 + r) * p.heads + h; }
  __device__ float query(int r, int c) const { return bf16_at(p.q + row(r) * (p.d + p.rope) + c); }
  __device__ int64_t last(int r) const { return first + r0 + r; }
  __device__ bool attends(int64_t pos) const { return pos < p.max_len; }
  __device__ void load(int64_t pos, float* k, float* v, int lane) const {
    const int64_t tok = (int64_t)b * p.max_len + pos;
    for (int c = lane; c < p.d; c += 32) {
      k[c] = pos < 0 ? 0.0f : bf16_at(p.k + tok * p.k_ts + h * p.k_hs + c);
      v[c] = pos < 0 ? 0.0f : bf16_at(p.v + tok * p.v_ts + h * p.v_hs + c);
    }
    for (int c = lane; c < p.rope; c += 32) k[p.d + c] = pos < 0 ? 0.0f : bf16_at(p.kr + tok * p.kr_ts + c);
  }
  __device__ void store(int r, int c, float x) const {
    const int64_t at = row(r) * p.d + c;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(x);
    else
      static_cast<float*>(p.out)[at] = x;
  }
};

__global__ void __launch_bounds__(kThreadsR) expanded_attn_kernel(const ExpandedParams p) {
  extern __shared__ float sm[];
  const int r0 = blockIdx.x % p.tiles * kRowsR, bh = blockIdx.x / p.tiles;
  const int h = bh % p.heads, b = bh / p.heads;
  const int32_t T = __ldg(p.lens + b), n = p.chunk_lens ? __ldg(p.chunk_lens + b) : p.chunk;
  if (n < 0 || n > p.chunk || T > p.max_len || T < n) {
    if (threadIdx.x == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
    if (n < 0 || n > p.chunk || T > p.max_len) return;
  }
  const int rows = min(kRowsR, n - r0);
  if (rows <= 0) return;
  ExpandedSrc src{p, b, h, r0, (int64_t)T - n};
  attend_rows(src, RowsShape{p.d + p.rope, p.d}, rows, T < n ? 0 : src.last(rows - 1) + 1, p.scale_log2, sm);
}

bool rows_ok(int64_t token, int64_t head, int64_t heads, int64_t width) {
  if (token % 8 != 0 || head % 8 != 0 || head < 0 || token < 0) return false;
  return (heads <= 1 || head >= width) && token >= (heads - 1) * head + width;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_expanded_attn(int32_t batch, int32_t num_heads, int32_t head_dim, int32_t rope_dim,
                                        int32_t chunk, int32_t max_len, const int32_t* d_seq_lens,
                                        const int32_t* d_chunk_lens, const void* q, const void* k,
                                        int64_t k_token_stride, int64_t k_head_stride, const void* k_rope,
                                        int64_t k_rope_stride, const void* v, int64_t v_token_stride,
                                        int64_t v_head_stride, float softmax_scale, void* out, int32_t out_dtype,
                                        int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 0 || num_heads < 1 || chunk < 0 || max_len < 0 || (head_dim != 64 && head_dim != 128) ||
      rope_dim != 64 || !(softmax_scale > 0.0f) || !(softmax_scale < INFINITY) ||
      (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (batch == 0 || chunk == 0) return KVQ_OK;
  if (d_seq_lens == nullptr || q == nullptr || out == nullptr || !aligned_to(q, 16) || !aligned_to(out, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (max_len > 0 && (k == nullptr || k_rope == nullptr || v == nullptr)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned_to(k, 16) || !aligned_to(k_rope, 16) || !aligned_to(v, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!rows_ok(k_token_stride, k_head_stride, num_heads, head_dim) || !rows_ok(k_rope_stride, 0, 1, rope_dim) ||
      !rows_ok(v_token_stride, v_head_stride, num_heads, head_dim))
    return KVQ_ERR_INVALID_ARGUMENT;
  if ((double)batch * chunk * num_heads > (double)(1 << 30)) return KVQ_ERR_UNSUPPORTED;
  ExpandedParams p = {};
  p.lens = d_seq_lens, p.chunk_lens = d_chunk_lens;
  p.q = static_cast<const uint16_t*>(q), p.k = static_cast<const uint16_t*>(k);
  p.kr = static_cast<const uint16_t*>(k_rope), p.v = static_cast<const uint16_t*>(v);
  p.out = out, p.flag = d_err_flag;
  p.k_ts = k_token_stride, p.k_hs = k_head_stride, p.kr_ts = k_rope_stride, p.v_ts = v_token_stride, p.v_hs = v_head_stride;
  p.batch = batch, p.heads = num_heads, p.d = head_dim, p.rope = rope_dim, p.chunk = chunk, p.max_len = max_len;
  p.out_bf16 = out_dtype == KVQ_DTYPE_BF16, p.tiles = (chunk + kRowsR - 1) / kRowsR;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  const size_t bytes = RowsShape{head_dim + rope_dim, head_dim}.bytes();
  if (cudaFuncSetAttribute(expanded_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
    return KVQ_ERR_CUDA;
  expanded_attn_kernel<<<(unsigned)((int64_t)batch * num_heads * p.tiles), kThreadsR, bytes,
                         reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}
