// kvq_block8.cuh -- the 8-bit paged cache (FP8 E4M3 codes, one fp32 scale per
// 16 tokens of one kv head): its pool layout, page lookup and host checks,
// shared by the append, dequantisation, decode and prefill kernels.
//
// One group = min(page_size, 64) tokens of one kv head, contiguous:
//   K codes [G/8][D/16][8][16]   8 tokens x 16 channels = one 128-byte core
//                                matrix of the tensor core's K-major layout
//   V codes [G/16][D][16]        per channel the 16 tokens of a block, in the
//                                order 0 1 8 9 2 3 10 11 4 5 12 13 6 7 14 15
//   scales  float [G/16][2]      (K, V), padded to 16 bytes
// Why: a 64-token decode stage is one bulk copy; ldmatrix reads both operands
// of the decode's products from it without bank conflicts (8 rows of 16
// contiguous bytes), and a V row of 16 bytes hands thread t the tokens 2t,
// 2t+1, 2t+8, 2t+9 it needs as one word; the K part of consecutive groups
// joins to one tensor-core operand without being touched.
#pragma once

#include "../../include/kvq_fp8_block.h"
#include "kvq_common.cuh"
#include "kvq_host.cuh"

namespace kvq {

struct Block8Layout {
  int D, P, G;
  __host__ __device__ Block8Layout(int head_dim, int page_size)
      : D(head_dim), P(page_size), G(page_size < 64 ? page_size : 64) {}
  __host__ __device__ int64_t group_bytes() const { return 2 * G * D + (G >= 32 ? G / 2 : 16); }
  __host__ __device__ int64_t page_bytes() const { return (P / G) * group_bytes(); }
  // byte offsets inside a group
  __host__ __device__ int k_code(int t, int c) const { return (t >> 3) * 8 * D + (c >> 4) * 128 + (t & 7) * 16 + (c & 15); }
  __host__ __device__ int v_row(int blk, int c) const { return G * D + (blk * D + c) * 16; }
  __host__ __device__ int scale(int blk, int side) const { return 2 * G * D + 8 * blk + 4 * side; }
};

// Byte of token u (0..15) of a block in a V row.
__host__ __device__ __forceinline__ int block8_v_byte(int u) {
  return u < 8 ? 4 * (u >> 1) + (u & 1) : 4 * ((u - 8) >> 1) + 2 + (u & 1);
}

// Physical page of position pos of sequence b, or -1 after setting PAGE_OOB.
__device__ __forceinline__ int64_t block8_page(const kvq_cache& c, int b, int64_t pos, int32_t* flag) {
  const int64_t pg = pos >> (__ffs(c.page_size) - 1);
  int64_t phys = -1;
  if (pg < c.max_pages_per_seq)
    phys = c.page_table ? (int64_t)__ldg(c.page_table + (int64_t)b * c.max_pages_per_seq + pg)
                        : (int64_t)b * c.max_pages_per_seq + pg;
  if (phys < 0 || phys >= c.num_pages) {
    set_flag(flag, KVQ_FLAG_PAGE_OOB);
    return -1;
  }
  return phys;
}

// The group of (physical page, kv head) that holds slot `slot` of the page.
__device__ __forceinline__ int64_t block8_group_offset(const Block8Layout& L, int64_t phys, int hkv, int h, int slot) {
  return (phys * hkv + h) * L.page_bytes() + (slot / L.G) * L.group_bytes();
}

inline kvq_status check_block8_cache(const kvq_cache* c, int32_t batch) {
  if (c == nullptr || c->reserved != 0 || c->format != KVQ_FORMAT_FP8_E4M3_BLOCK) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->num_kv_heads < 1 || c->data == nullptr || !aligned_to(c->data, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 64 && c->head_dim != 128) return KVQ_ERR_INVALID_ARGUMENT;
  if (!is_pow2_page(c->page_size) || c->num_pages < 1 || c->max_pages_per_seq < 1) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->v_data != nullptr || c->k_scale != nullptr || c->v_scale != nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->page_table != nullptr && !aligned_to(c->page_table, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->page_table == nullptr && (int64_t)batch * c->max_pages_per_seq > c->num_pages) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->num_pages > (int64_t)INT32_MAX / c->num_kv_heads) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

}  // namespace kvq
