// kvq_latent_attn.cu -- attention over the latent cache (absorbed form), one
// token per sequence or a chunk of them, and its C entry points.
//   y = softmax_scale log2 e (q . [c, k]),  out = sum 2^(y - m) c / sum 2^(y - m)
// with the tokens' values as the cache holds them.
#include "kvq_attn_rows.cuh"
#include "kvq_latent.cuh"

#include <cuda_bf16.h>

namespace kvq {
namespace {

struct LatentAttnParams {
  kvq_latent_cache c;
  const int32_t* lens;
  const int32_t* chunk_lens;
  const uint16_t* q;
  void* out;
  int32_t* flag;
  int32_t batch, hq, chunk, out_bf16, tiles;
  float scale_log2;
};

struct LatentSrc {
  const LatentAttnParams& p;
  LatentLayout lay;
  int b, r0;
  int64_t first;  // position of the chunk's token 0
  __device__ int64_t row(int r) const { return (int64_t)b * p.chunk * p.hq + r0 + r; }
  __device__ float query(int r, int c) const {
    return __uint_as_float((uint32_t)p.q[row(r) * (lay.L + lay.R) + c] << 16);
  }
  __device__ int64_t last(int r) const { return first + (r0 + r) / p.hq; }
  __device__ int64_t group(int64_t pos, int32_t* flag) const { return latent_group(p.c, lay, b, pos, flag); }
  __device__ bool attends(int64_t pos) const { return pos >= 0 && pos <= first + p.chunk && group(pos, p.flag) >= 0; }
  __device__ void load(int64_t pos, float* k, float* v, int lane) const {
    const int64_t grp = pos < 0 ? -1 : group(pos, p.flag);
    const uint8_t* base = static_cast<const uint8_t*>(p.c.data) + grp;
    const int slot = (int)(pos & (lay.G - 1));
    const float s = grp < 0 ? 0.0f : latent_scale(base[lay.exponent(slot)]);
    for (int c = lane; c < lay.L + lay.R; c += 32) {
      float x = 0.0f;
      if (grp >= 0) {
        x = e4m3_to_f32(base[lay.unit(slot, c >> 4) + (c & 15)]);
        if (c >= lay.L) x += e4m3_to_f32(base[lay.unit(slot, (c + lay.R) >> 4) + (c & 15)]);
        x *= s;
      }
      k[c] = x;
      if (c < lay.L) v[c] = x;
    }
  }
  __device__ void store(int r, int c, float x) const {
    const int64_t at = row(r) * lay.L + c;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(x);
    else
      static_cast<float*>(p.out)[at] = x;
  }
};

__global__ void __launch_bounds__(kThreadsR) latent_attn_kernel(const LatentAttnParams p) {
  extern __shared__ float sm[];
  const int b = blockIdx.x / p.tiles, r0 = blockIdx.x % p.tiles * kRowsR;
  const int32_t T = __ldg(p.lens + b), n = p.chunk_lens ? __ldg(p.chunk_lens + b) : p.chunk;
  const bool decode = p.chunk == 1 && p.chunk_lens == nullptr;
  if (n < 0 || n > p.chunk || T < (decode ? 0 : n)) {
    if (threadIdx.x == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
    if (n < 0 || n > p.chunk) return;
  }
  const int rows = min(kRowsR, n * p.hq - r0);
  if (rows <= 0) return;
  LatentSrc src{p, LatentLayout(p.c), b, r0, (int64_t)T - n};
  const int64_t cap = (int64_t)p.c.max_pages_per_seq * p.c.page_size;
  int64_t limit = T < n ? 0 : src.last(rows - 1) + 1;
  if (limit > cap) {
    if (threadIdx.x == 0) set_flag(p.flag, KVQ_FLAG_PAGE_OOB);
    limit = cap;
  }
  attend_rows(src, RowsShape{p.c.latent_dim + p.c.rope_dim, p.c.latent_dim}, rows, limit, p.scale_log2, sm);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_latent_attn_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t latent_dim,
                                                  int32_t chunk) {
  if (batch < 1 || num_q_heads < 1 || chunk < 1 || !latent_dims_ok(16, latent_dim, 64)) return 0;
  return 16;
}

extern "C" kvq_status kvq_latent_attn(const kvq_latent_cache* cache, int32_t batch, int32_t num_q_heads, int32_t chunk,
                                      const int32_t* d_seq_lens, const int32_t* d_chunk_lens, const void* q,
                                      float softmax_scale, void* out, int32_t out_dtype, void* workspace,
                                      size_t workspace_bytes, int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 0 || num_q_heads < 1 || chunk < 0 || !(softmax_scale > 0.0f) || !(softmax_scale < INFINITY) ||
      (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_status st = check_latent_cache(cache, batch);
  if (st != KVQ_OK) return st;
  if (batch == 0 || chunk == 0) return KVQ_OK;
  if (d_seq_lens == nullptr || q == nullptr || out == nullptr || workspace == nullptr || !aligned_to(q, 16) ||
      !aligned_to(out, 16) || !aligned_to(workspace, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  if ((double)batch * chunk * num_q_heads > (double)(1 << 30)) return KVQ_ERR_UNSUPPORTED;
  if (workspace_bytes < kvq_latent_attn_workspace_bytes(batch, num_q_heads, cache->latent_dim, chunk))
    return KVQ_ERR_WORKSPACE;
  LatentAttnParams p = {};
  p.c = *cache;
  p.lens = d_seq_lens, p.chunk_lens = d_chunk_lens;
  p.q = static_cast<const uint16_t*>(q), p.out = out, p.flag = d_err_flag;
  p.batch = batch, p.hq = num_q_heads, p.chunk = chunk, p.out_bf16 = out_dtype == KVQ_DTYPE_BF16;
  p.tiles = (int32_t)(((int64_t)chunk * num_q_heads + kRowsR - 1) / kRowsR);
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  const size_t bytes = RowsShape{cache->latent_dim + cache->rope_dim, cache->latent_dim}.bytes();
  if (cudaFuncSetAttribute(latent_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
    return KVQ_ERR_CUDA;
  latent_attn_kernel<<<(unsigned)(batch * p.tiles), kThreadsR, bytes, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}
