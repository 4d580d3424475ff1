// kvq_block8_dequant.cu -- dense values of the 8-bit block cache.
//
// value = fp32(E4M3(code) * scale), the scale shared by the 16 tokens of a
// block of one kv head.  One thread per 16 channels of one token: a K item is one
// 16-byte read; the V bytes of a token lie 16 apart, so a thread reads single bytes
// and each of a block's 16 tokens, num_kv_heads * head_dim / 16 threads apart, reads
// the same 256 bytes again, from L1 or L2.  Lanes run over the channels first, so the
// stores of a row are contiguous.  By its bytes HBM would bound it (one read per 2 or
// 4 written); measured, 8 x 8192 positions of 8 heads of 128: 158 us to bf16, 2.56
// TB/s (0.38 of the copy rate), 229 us to fp32, 2.93 TB/s (0.43).
#include <cuda_bf16.h>

#include "kvq_block8.cuh"

namespace kvq {
namespace {

__device__ __forceinline__ void store_values(void* out, int64_t elem, const float (&x)[16], int dtype) {
  if (dtype == KVQ_DTYPE_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + elem);
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
    return;
  }
  uint32_t w[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
    w[q] = *reinterpret_cast<const uint32_t*>(&p);
  }
  uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + elem);
  o[0] = make_uint4(w[0], w[1], w[2], w[3]);
  o[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__global__ void __launch_bounds__(256) dequant_block8_kernel(const kvq_cache c, int32_t batch,
                                                             const int32_t* __restrict__ lens, int32_t max_len,
                                                             int dtype, void* k_out, void* v_out, int32_t* flag) {
  const int nblk = c.head_dim >> 4, hkv = c.num_kv_heads;
  const Block8Layout L(c.head_dim, c.page_size);
  const int64_t total = (int64_t)batch * max_len * hkv * nblk;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int c0 = 16 * (int)(i % nblk);
    int64_t r = i / nblk;
    const int h = (int)(r % hkv);
    r /= hkv;
    const int pos = (int)(r % max_len), b = (int)(r / max_len);
    const int32_t len = __ldg(lens + b);
    if (len < 0) set_flag(flag, KVQ_FLAG_BAD_LENGTH);
    float kx[16], vx[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) kx[q] = vx[q] = 0.0f;
    const int64_t phys = pos < len ? block8_page(c, b, pos, flag) : -1;
    if (phys >= 0) {
      const int slot = pos & (c.page_size - 1), lt = slot & (L.G - 1);
      const int64_t off = block8_group_offset(L, phys, hkv, h, slot);
      if (KVQ_IN(off >= 0 && off + L.group_bytes() <= c.num_pages * (int64_t)hkv * L.page_bytes(), flag)) {
        const uint8_t* grp = static_cast<const uint8_t*>(c.data) + off;
        const float2 s = __ldg(reinterpret_cast<const float2*>(grp + L.scale(lt >> 4, 0)));
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(grp + L.k_code(lt, c0)));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        const uint8_t* vr = grp + L.v_row(lt >> 4, c0) + block8_v_byte(lt & 15);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 f = f16x2_to_float2(f16x2_from_e4m3x2((ws[q >> 1] >> (16 * (q & 1))) & 0xFFFFu));
          kx[2 * q] = f.x * s.x;
          kx[2 * q + 1] = f.y * s.x;
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) vx[q] = e4m3_to_f32(__ldg(vr + 16 * q)) * s.y;
      }
    }
    store_values(k_out, i * 16, kx, dtype);
    store_values(v_out, i * 16, vx, dtype);
  }
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_fp8_block_dequant(const kvq_cache* cache, int32_t batch, const int32_t* d_seq_lens,
                                            int32_t max_len, int32_t out_dtype, void* k_out, void* v_out,
                                            int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 0 || max_len < 0 || (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_status st = check_block8_cache(cache, batch);
  if (st != KVQ_OK) return st;
  if (batch == 0 || max_len == 0) return KVQ_OK;
  if (d_seq_lens == nullptr || k_out == nullptr || v_out == nullptr || !aligned_to(k_out, 16) || !aligned_to(v_out, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  const int64_t work = (int64_t)batch * max_len * cache->num_kv_heads * (cache->head_dim / 16);
  dequant_block8_kernel<<<grid_for(work, 256), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      *cache, batch, d_seq_lens, max_len, out_dtype, k_out, v_out, d_err_flag);
  return launch_status();
}
