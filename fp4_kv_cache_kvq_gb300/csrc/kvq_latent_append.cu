// kvq_latent_append.cu -- the latent cache's append (rotation of the key and
// query parts, quantisation, paged store) and its dense read-back, with their C
// entry points.
//
// Append: y = rot(k), s = 2^e the smallest power of two with max(|c|, |y|) <=
// 448 s, codes E4M3(c / s), hi = E4M3(y / s), lo = E4M3(y / s - hi).  s is a power
// of two, so x / s is exact and every code is one rounding; y has 8 significant
// bits (bf16), of which hi takes 4, so y / s - hi is exact too.
// Both are bound by HBM: 2 (L + R) bytes in and L + 2 R + 1 out per token, 4 R per
// query head.
#include "kvq_latent.cuh"

namespace kvq {
namespace {

constexpr int kThreadsA = 256;
constexpr int kThreadsD = 8 * (512 + 64) / 16;  // of the read-back, at most
constexpr int kQHeads = 2;  // query heads of a thread: they share the angles
constexpr uint32_t kInfBits = 0x7F800000u;

struct LatentAppendParams {
  kvq_latent_cache c;
  const int32_t* start;
  const int32_t* new_lens;
  const uint16_t* q;
  const uint16_t* lat;
  const uint16_t* k;
  const float* table;
  uint16_t* q_out;
  uint16_t* k_out;
  int32_t* flag;
  int64_t q_ts, q_hs, qo_ts, qo_hs, c_ts, k_ts, table_rows;
  int32_t batch, n_new, hq, interleaved;
  uint32_t blocks;   // 8-token blocks per sequence
  uint32_t head_groups;  // of kQHeads query heads
  uint32_t tok_ctas;     // CTAs of latents and key parts; the rest rotate queries
};

// New tokens of sequence b and its start; 0 tokens (flagged) where either is bad.
__device__ __forceinline__ int new_tokens(const LatentAppendParams& p, int b, int32_t& sp) {
  sp = __ldg(p.start + b);
  const int n = p.new_lens ? __ldg(p.new_lens + b) : p.n_new;
  if (sp < 0 || n < 0 || n > p.n_new) {
    set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
    return 0;
  }
  return n;
}

// Two fp32 values rounded to bf16 (lo in the low half).
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight cosines, then eight sines, `half` behind them in the table's row.
__device__ __forceinline__ void load_angles(const float* row, int half, float (&cs)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(row + (i >> 1) * half) + (i & 1));
    cs[4 * i] = v.x, cs[4 * i + 1] = v.y, cs[4 * i + 2] = v.z, cs[4 * i + 3] = v.w;
  }
}

// Eight pairs: a and b hold the first and the second halves' 8 values (or, of
// adjacent pairs, 16 consecutive values); rotated in place.  Every product and sum
// is rounded to fp32, the result to bf16.
__device__ __forceinline__ void rotate8(uint4& a, uint4& b, const float (&cs)[16], int interleaved) {
  uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  const auto turn = [&](float x0, float x1, int i, float& y0, float& y1) {
    y0 = __fsub_rn(__fmul_rn(x0, cs[i]), __fmul_rn(x1, cs[8 + i]));
    y1 = __fadd_rn(__fmul_rn(x1, cs[i]), __fmul_rn(x0, cs[8 + i]));
  };
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0, y1;
      turn(bf16_lo(wa[i]), bf16_hi(wa[i]), i, y0, y1);
      wa[i] = bf16x2_rn(y0, y1);
      turn(bf16_lo(wb[i]), bf16_hi(wb[i]), 4 + i, y0, y1);
      wb[i] = bf16x2_rn(y0, y1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u0, u1, v0, v1;
      turn(bf16_lo(wa[i]), bf16_lo(wb[i]), 2 * i, u0, u1);
      turn(bf16_hi(wa[i]), bf16_hi(wb[i]), 2 * i + 1, v0, v1);
      wa[i] = bf16x2_rn(u0, v0);
      wb[i] = bf16x2_rn(u1, v1);
    }
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

// Largest magnitude of 8 bf16 values, as fp32 bits (NaN above Inf above the rest).
__device__ __forceinline__ uint32_t amax8(uint4 v) {
  uint32_t m = 0u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] << 16 & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
  return m;
}

// Exponent byte of a token with this largest magnitude (finite, as fp32 bits).
__device__ __forceinline__ uint32_t exponent_of(uint32_t amax) {
  const int x = (int)(amax >> 23);                                     // amax = 1.f 2^(x - 127), 448 = 1.75 2^8
  const int e = x - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}

// 8 values times mul as 8 E4M3 codes.
__device__ __forceinline__ uint2 encode8(uint4 v, float mul) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x2_from_f32(bf16_lo(w[i]) * mul, bf16_hi(w[i]) * mul);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// ... and as hi and lo codes.
__device__ __forceinline__ void encode8_split(uint4 v, float mul, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = bf16_lo(w[i]) * mul, x1 = bf16_hi(w[i]) * mul;
    h[i] = e4m3x2_from_f32(x0, x1);
    const float2 y = f16x2_to_float2(f16x2_from_e4m3x2(h[i]));
    l[i] = e4m3x2_from_f32(x0 - y.x, x1 - y.y);
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

__device__ __forceinline__ uint4 ldg128(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Channel offsets of the two 8-value pieces of rotation item i of a head.
__device__ __forceinline__ int piece_a(int i, int interleaved) { return interleaved ? 16 * i : 8 * i; }
__device__ __forceinline__ int piece_b(int i, int half, int interleaved) { return interleaved ? 16 * i + 8 : half + 8 * i; }

// One 8-token block of a sequence (aligned to positions) takes L/2 threads: thread
// (token t = lane & 7, unit u) 16 channels of the latent, so that 8 lanes store one
// core matrix; the block's first warp also takes the key parts, lane (t, item).
template <int L>
__global__ void __launch_bounds__(kThreadsA, 5) latent_append_kernel(const LatentAppendParams p) {
  constexpr int kPer = L / 2, kBlocks = kThreadsA / kPer;
  __shared__ uint32_t amax_s[kBlocks * 8];
  const int tid = threadIdx.x, R = p.c.rope_dim, half = R / 2;
  if (blockIdx.x >= p.tok_ctas) {  // query parts: eight pairs of kQHeads heads a thread
    const uint32_t i = (blockIdx.x - p.tok_ctas) * kThreadsA + tid;  // under 2^30 + 256
    const uint32_t it = i & ((uint32_t)R / 16u - 1u), rest = i >> (R == 64 ? 2 : 1);
    const uint32_t tok32 = rest / p.head_groups;
    const int h0 = (int)(rest - tok32 * p.head_groups) * kQHeads, heads = min(kQHeads, p.hq - h0);
    const int b = (int)(tok32 / (uint32_t)p.n_new), t = (int)(tok32 - (uint32_t)b * (uint32_t)p.n_new);
    if (b >= p.batch) return;
    const int64_t tok = tok32;
    const uint16_t* src = p.q + tok * p.q_ts + h0 * p.q_hs;
    uint16_t* dst = p.q_out + tok * p.qo_ts + h0 * p.qo_hs;
    const int ca = piece_a(it, p.interleaved), cb = piece_b(it, half, p.interleaved);
    int32_t sp;
    if (t >= new_tokens(p, b, sp)) return;
    uint4 va[kQHeads], vb[kQHeads];
#pragma unroll
    for (int k = 0; k < kQHeads; ++k)
      if (k < heads) {
        va[k] = *reinterpret_cast<const uint4*>(src + k * p.q_hs + ca);
        vb[k] = *reinterpret_cast<const uint4*>(src + k * p.q_hs + cb);
      }
    float cs[16];
    const int64_t pos = (int64_t)sp + t;
    if (p.table != nullptr) {
      if (pos >= p.table_rows) {
        set_flag(p.flag, KVQ_FLAG_POSITION);
        return;
      }
      load_angles(p.table + pos * R + 8 * it, half, cs);
    }
#pragma unroll
    for (int k = 0; k < kQHeads; ++k)
      if (k < heads) {
        if (p.table != nullptr) rotate8(va[k], vb[k], cs, p.interleaved);
        *reinterpret_cast<uint4*>(dst + k * p.qo_hs + ca) = va[k];
        *reinterpret_cast<uint4*>(dst + k * p.qo_hs + cb) = vb[k];
      }
    return;
  }
  if (tid < kBlocks * 8) amax_s[tid] = 0u;
  __syncthreads();
  const uint32_t blk = blockIdx.x * kBlocks + tid / kPer;
  const int b = (int)(blk / p.blocks), j = (int)(blk % p.blocks);
  const int lane = tid & 31, t8 = lane & 7, u = (tid % kPer) / 32 * 4 + (lane >> 3);
  const bool rope = tid % kPer < 32 && (lane >> 3) < R / 16;
  int32_t sp = 0;
  const int n = b < p.batch ? new_tokens(p, b, sp) : 0;
  const int t = j * 8 + t8 - (sp & 7);
  const int64_t pos = (int64_t)sp + t;
  bool ok = t >= 0 && t < n;
  if (ok && p.table != nullptr && pos >= p.table_rows) {
    set_flag(p.flag, KVQ_FLAG_POSITION);
    ok = false;
  }
  const int64_t tok = (int64_t)b * p.n_new + t;
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0, ka = v0, kb = v0;
  const int it = lane >> 3, ca = piece_a(it, p.interleaved), cb = piece_b(it, half, p.interleaved);
  const LatentLayout lay(p.c);
  int64_t grp = -1;
  if (ok) {
    const uint16_t* src = p.lat + tok * p.c_ts + 16 * u;
    v0 = ldg128(src);
    v1 = ldg128(src + 8);
    if (rope) {
      ka = *reinterpret_cast<const uint4*>(p.k + tok * p.k_ts + ca);
      kb = *reinterpret_cast<const uint4*>(p.k + tok * p.k_ts + cb);
    }
    grp = latent_group(p.c, lay, b, pos, p.flag);
    if (rope && p.table != nullptr) {
      float cs[16];
      load_angles(p.table + pos * R + 8 * it, half, cs);
      rotate8(ka, kb, cs, p.interleaved);
    }
  }
  uint32_t m = max(max(amax8(v0), amax8(v1)), max(amax8(ka), amax8(kb)));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
  uint32_t* amax = amax_s + tid / kPer * 8;
  if (lane < 8) atomicMax(amax + t8, m);
  __syncthreads();
  if (!ok) return;
  if (rope && p.k_out != nullptr) {
    *reinterpret_cast<uint4*>(p.k_out + tok * R + ca) = ka;
    *reinterpret_cast<uint4*>(p.k_out + tok * R + cb) = kb;
  }
  m = amax[t8];
  uint32_t e = 255u;  // a token with Inf or NaN: marked, codes 0
  if (m < kInfBits) {
    e = exponent_of(m);
  } else {
    if (u == 0) set_flag(p.flag, KVQ_FLAG_NONFINITE);
    v0 = v1 = ka = kb = make_uint4(0u, 0u, 0u, 0u);
  }
  if (grp < 0) return;
  if (!KVQ_IN(grp + lay.group_bytes() <= p.c.num_pages * lay.page_bytes(), p.flag)) return;
  const float mul = e == 255u ? 1.0f : __uint_as_float((254u - e) << 23);
  uint8_t* base = static_cast<uint8_t*>(p.c.data) + grp;
  const int slot = (int)(pos & (lay.G - 1));
  const uint2 w0 = encode8(v0, mul), w1 = encode8(v1, mul);
  *reinterpret_cast<uint4*>(base + lay.unit(slot, u)) = make_uint4(w0.x, w0.y, w1.x, w1.y);
  if (u == 0) base[lay.exponent(slot)] = (uint8_t)e;
  if (rope) {
    uint2 ha, la, hb, lb;
    encode8_split(ka, mul, ha, la);
    encode8_split(kb, mul, hb, lb);
    const int ua = L + ca, ub = L + cb;  // channels of a token's row
    *reinterpret_cast<uint2*>(base + lay.unit(slot, ua >> 4) + (ua & 15)) = ha;
    *reinterpret_cast<uint2*>(base + lay.unit(slot, ub >> 4) + (ub & 15)) = hb;
    *reinterpret_cast<uint2*>(base + lay.unit(slot, (ua + R) >> 4) + (ua & 15)) = la;
    *reinterpret_cast<uint2*>(base + lay.unit(slot, (ub + R) >> 4) + (ub & 15)) = lb;
  }
}

struct LatentDequantParams {
  kvq_latent_cache c;
  const int32_t* lens;
  void* c_out;
  void* k_out;
  int32_t* flag;
  int32_t batch, max_len;
  uint32_t pairs;  // pairs of 8-token blocks per sequence
};

// 16 E4M3 codes (bytes of v) as fp32.
__device__ __forceinline__ void decode16(uint4 v, float (&x)[16]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f16x2_to_float2(f16x2_from_e4m3x2(w[i])), b = f16x2_to_float2(f16x2_from_e4m3x2(w[i] >> 16));
    x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
  }
}

__device__ __forceinline__ void store16(float* dst, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(uint16_t* dst, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = bf16x2_rn(x[2 * i], x[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// A CTA takes two blocks of 8 tokens, a thread one token's 16 channels (of the latent,
// then of the key part) in each, 8 tokens side by side in a warp: they read one core
// matrix.
template <typename T>
__global__ void __launch_bounds__(kThreadsD) latent_dequant_kernel(const LatentDequantParams p) {
  const LatentLayout lay(p.c);
  const uint32_t pair = blockIdx.x % p.pairs;
  const int b = (int)(blockIdx.x / p.pairs), t8 = threadIdx.x & 7, u = threadIdx.x >> 3;
  const int len = __ldg(p.lens + b);
  if (len < 0 && pair == 0 && threadIdx.x == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
  const bool key = 16 * u >= lay.L;
  const uint8_t* pool = static_cast<const uint8_t*>(p.c.data);
  uint4 v[2], w[2];
  uint32_t e[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t pos = (int64_t)pair * 16 + 8 * i + t8;
    v[i] = w[i] = make_uint4(0u, 0u, 0u, 0u);
    e[i] = 1u;
    if (pos >= len || pos >= p.max_len) continue;
    const int64_t grp = latent_group(p.c, lay, b, pos, p.flag);
    if (grp < 0 || !KVQ_IN(grp + lay.group_bytes() <= p.c.num_pages * lay.page_bytes(), p.flag)) continue;
    const int slot = (int)(pos & (lay.G - 1));
    e[i] = __ldg(pool + grp + lay.exponent(slot));
    v[i] = __ldg(reinterpret_cast<const uint4*>(pool + grp + lay.unit(slot, u)));
    if (key) w[i] = __ldg(reinterpret_cast<const uint4*>(pool + grp + lay.unit(slot, u + lay.R / 16)));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t pos = (int64_t)pair * 16 + 8 * i + t8;
    if (pos >= p.max_len) continue;
    float x[16];
    decode16(v[i], x);
    if (key) {
      float lo[16];
      decode16(w[i], lo);
#pragma unroll
      for (int c = 0; c < 16; ++c) x[c] += lo[c];
    }
    const float s = latent_scale(e[i]);
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] *= s;
    const int64_t row = (int64_t)b * p.max_len + pos;
    if (!key)
      store16(static_cast<T*>(p.c_out) + row * lay.L + 16 * u, x);
    else
      store16(static_cast<T*>(p.k_out) + row * lay.R + 16 * u - lay.L, x);
  }
}

// Strides of rows of `width` values: multiples of 8 that leave no overlap.
bool strides_ok(int64_t token, int64_t head, int64_t heads, int64_t width) {
  if (token % 8 != 0 || head % 8 != 0 || head < 0 || token < 0) return false;
  return (heads <= 1 || head >= width) && token >= (heads - 1) * head + width;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_latent_pool_bytes(int64_t num_pages, int32_t page_size, int32_t latent_dim, int32_t rope_dim) {
  if (num_pages < 0 || num_pages > INT32_MAX || !latent_dims_ok(page_size, latent_dim, rope_dim)) return 0;
  kvq_latent_cache c = {};
  c.latent_dim = latent_dim, c.rope_dim = rope_dim, c.page_size = page_size;
  return (size_t)num_pages * (size_t)LatentLayout(c).page_bytes();
}

extern "C" kvq_status kvq_latent_append(const kvq_latent_cache* cache, int32_t batch, int32_t n_new,
                                        const int32_t* d_start_pos, const int32_t* d_new_lens, int32_t num_q_heads,
                                        const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* c,
                                        int64_t c_stride, const void* k, int64_t k_stride, const float* table,
                                        int64_t table_rows, int32_t interleaved, void* q_out,
                                        int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                                        int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 0 || n_new < 0 || num_q_heads < 0) return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_status st = check_latent_cache(cache, batch);
  if (st != KVQ_OK) return st;
  const int32_t L = cache->latent_dim, R = cache->rope_dim;
  if ((interleaved != 0 && interleaved != 1) || table_rows < 0 || (table == nullptr && table_rows != 0) ||
      !aligned_to(table, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (batch == 0 || n_new == 0) return KVQ_OK;
  if (d_start_pos == nullptr || c == nullptr || k == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if ((num_q_heads > 0) != (q != nullptr) || (num_q_heads > 0) != (q_out != nullptr)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned_to(q, 16) || !aligned_to(c, 16) || !aligned_to(k, 16) || !aligned_to(q_out, 16) || !aligned_to(k_out, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!strides_ok(c_stride, 0, 1, L) || !strides_ok(k_stride, 0, 1, R)) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads > 0 && (!strides_ok(q_token_stride, q_head_stride, num_q_heads, R) ||
                          !strides_ok(q_out_token_stride, q_out_head_stride, num_q_heads, R)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads > 0 && q_out == q &&
      (q_out_token_stride != q_token_stride || (num_q_heads > 1 && q_out_head_stride != q_head_stride)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (k_out == k || k_out == c) {
    if (k_out != nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  }
  LatentAppendParams p = {};
  p.c = *cache;
  p.start = d_start_pos, p.new_lens = d_new_lens;
  p.q = static_cast<const uint16_t*>(q), p.lat = static_cast<const uint16_t*>(c);
  p.k = static_cast<const uint16_t*>(k), p.table = table;
  p.q_out = static_cast<uint16_t*>(q_out), p.k_out = static_cast<uint16_t*>(k_out), p.flag = d_err_flag;
  p.q_ts = q_token_stride, p.q_hs = q_head_stride, p.qo_ts = q_out_token_stride, p.qo_hs = q_out_head_stride;
  p.c_ts = c_stride, p.k_ts = k_stride, p.table_rows = table_rows;
  p.batch = batch, p.n_new = n_new, p.hq = num_q_heads, p.interleaved = interleaved;
  p.blocks = ((uint32_t)n_new + 14u) / 8u;  // aligned blocks can be cut at both ends
  const double tok = (double)batch * p.blocks * (L / 2), qi = (double)batch * n_new * ((num_q_heads + kQHeads - 1) / kQHeads) * (R / 16);
  if (tok > (double)(1 << 30) || qi > (double)(1 << 30)) return KVQ_ERR_UNSUPPORTED;
  p.head_groups = (uint32_t)((num_q_heads + kQHeads - 1) / kQHeads);
  p.tok_ctas = grid_for((int64_t)tok, kThreadsA);
  const unsigned grid = p.tok_ctas + (num_q_heads > 0 ? grid_for((int64_t)qi, kThreadsA) : 0u);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (L == 128)
    latent_append_kernel<128><<<grid, kThreadsA, 0, s>>>(p);
  else if (L == 256)
    latent_append_kernel<256><<<grid, kThreadsA, 0, s>>>(p);
  else
    latent_append_kernel<512><<<grid, kThreadsA, 0, s>>>(p);
  return launch_status();
}

extern "C" kvq_status kvq_latent_dequant(const kvq_latent_cache* cache, int32_t batch, const int32_t* d_seq_lens,
                                         int32_t max_len, int32_t out_dtype, void* c_out, void* k_out,
                                         int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 0 || max_len < 0 || (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_status st = check_latent_cache(cache, batch);
  if (st != KVQ_OK) return st;
  if (batch == 0 || max_len == 0) return KVQ_OK;
  if (d_seq_lens == nullptr || c_out == nullptr || k_out == nullptr || !aligned_to(c_out, 16) || !aligned_to(k_out, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  LatentDequantParams p = {};
  p.c = *cache;
  p.lens = d_seq_lens;
  p.c_out = c_out, p.k_out = k_out, p.flag = d_err_flag;
  p.batch = batch, p.max_len = max_len;
  p.pairs = ((uint32_t)max_len + 15u) / 16u;
  if ((double)batch * p.pairs > 2147483647.0) return KVQ_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)batch * p.pairs, threads = 8u * (unsigned)(cache->latent_dim + cache->rope_dim) / 16u;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (out_dtype == KVQ_DTYPE_BF16)
    latent_dequant_kernel<uint16_t><<<grid, threads, 0, s>>>(p);
  else
    latent_dequant_kernel<float><<<grid, threads, 0, s>>>(p);
  return launch_status();
}
