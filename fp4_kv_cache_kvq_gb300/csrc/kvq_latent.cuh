// kvq_latent.cuh -- the latent cache (E4M3 codes of one latent vector and of one
// rotated key part per token, an exponent byte per token): its pool layout, page
// lookup and host checks, shared by the append, dequantisation and attention
// kernels.
//
// One group = min(page_size, 64) tokens, contiguous: codes [G/8][row/16][8][16],
// row = latent + 2 rope bytes, then the exponents [G].  8 tokens x 16 channels
// are one 128-byte core matrix of the tensor core.  Read with tokens as rows it
// is a K-major operand (scores: the sum runs over channels); read with channels
// as rows it is an MN-major one (the sum runs over tokens).  So one copy of a
// tile in shared memory serves both products untouched.
#pragma once

#include "../../include/kvq_latent.h"
#include "kvq_common.cuh"
#include "kvq_host.cuh"

namespace kvq {

struct LatentLayout {
  int L, R, P, G;
  __host__ __device__ explicit LatentLayout(const kvq_latent_cache& c)
      : L(c.latent_dim), R(c.rope_dim), P(c.page_size), G(c.page_size < 64 ? c.page_size : 64) {}
  __host__ __device__ int row() const { return L + 2 * R; }
  __host__ __device__ int group_bytes() const { return G * row() + G; }
  __host__ __device__ int64_t page_bytes() const { return (int64_t)(P / G) * group_bytes(); }
  // byte offsets inside a group: 16-byte unit u of token t, and its exponent
  __host__ __device__ int unit(int t, int u) const { return (t >> 3) * 8 * row() + u * 128 + (t & 7) * 16; }
  __host__ __device__ int exponent(int t) const { return G * row() + t; }
};

// Byte offset in the pool of the group that holds position pos of sequence b,
// or -1 after setting PAGE_OOB.
__device__ __forceinline__ int64_t latent_group(const kvq_latent_cache& c, const LatentLayout& L, int b, int64_t pos,
                                                int32_t* flag) {
  const int64_t pg = pos >> (__ffs(c.page_size) - 1);
  int64_t phys = -1;
  if (pg < c.max_pages_per_seq)
    phys = c.page_table ? (int64_t)__ldg(c.page_table + (int64_t)b * c.max_pages_per_seq + pg)
                        : (int64_t)b * c.max_pages_per_seq + pg;
  if (phys < 0 || phys >= c.num_pages) {
    set_flag(flag, KVQ_FLAG_PAGE_OOB);
    return -1;
  }
  return phys * L.page_bytes() + (int64_t)((int)(pos & (c.page_size - 1)) / L.G) * L.group_bytes();
}

// A token's scale of its exponent byte; 255 (a token that held Inf or NaN): NaN.
__device__ __forceinline__ float latent_scale(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7FFFFFFFu : e << 23);
}

inline bool latent_dims_ok(int32_t page_size, int32_t latent_dim, int32_t rope_dim) {
  return (latent_dim == 128 || latent_dim == 256 || latent_dim == 512) && (rope_dim == 32 || rope_dim == 64) &&
         is_pow2_page(page_size);
}

inline kvq_status check_latent_cache(const kvq_latent_cache* c, int32_t batch) {
  if (c == nullptr || !latent_dims_ok(c->page_size, c->latent_dim, c->rope_dim)) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->data == nullptr || !aligned_to(c->data, 16) || c->num_pages < 1 || c->max_pages_per_seq < 1)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (c->page_table != nullptr && !aligned_to(c->page_table, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->page_table == nullptr && (int64_t)batch * c->max_pages_per_seq > c->num_pages) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->num_pages > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

}  // namespace kvq
