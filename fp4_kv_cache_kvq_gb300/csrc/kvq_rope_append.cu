// kvq_rope_append.cu -- the append with the rotary position embedding on the
// way: queries and keys rotated by their positions, keys and values quantised
// into the 8-bit block cache or the FP4 / NVFP4 caches, in one launch; the
// same kernel without a rotation is the 8-bit cache's plain append.
//
// Mathematics.  Pair (x0, x1) of a token at position p with frequency i:
//   y0 = x0 cos(p w_i) - x1 sin(p w_i),  y1 = x1 cos(p w_i) + x0 sin(p w_i)
// with each product and sum rounded to fp32 (no contraction, so the result
// does not depend on how a compiler fuses it) and the result rounded to bf16:
// that rounding (at most half a step, 2^-9 relative, far under the codes' own
// 2^-4) keeps one definition for a rotated key, whether it is rotated here or
// beforehand.  cos and sin come from a table that every head of a token
// shares.  8-bit block: s = 2^e, the smallest with amax <= 448 * 2^e, so x / s
// is exact and only the E4M3 conversion rounds, and raising s later moves
// kept codes by a power of two, again exact outside the subnormals.
//
// Measured: 8 prompts of 4096 tokens, 64 query and 8 kv heads of 128, 8 bit:
// 204 us, 6.27 TB/s (1.28 GB: 0.93 of the copy rate); FP4, 32 query heads: 124 us,
// 5.73 TB/s.  Four CTAs of 8 warps per SM (64 registers) against two: 226 -> 211 us;
// the input's loads issued ahead of the page table's and bf16 quotients two at a
// time: 211 -> 204.
//
// What bounds it: HBM.  Per token 2 * Hq * d bf16 values move for the queries
// and Hkv * d * (2 + 1) bytes for each of K and V; a table row is read once per 16
// heads from L1/L2.  Work is cut into warp tasks, one memory round trip each:
//   K, 8 bit   a 16-token block of two kv heads by a group of D/32 warps: a lane
//              holds one token's chunks of both heads, so its angles are read
//              once; the blocks' maxima meet in shared memory (16 x 4096 tokens,
//              8 kv and 8 query heads of 128: one head per group 158 us, two
//              136, four 141 with spills)
//   V, 8 bit   the block of one kv head by a warp; a lane holds D/32 channels of
//              all 16 tokens, so the codes of a channel are 16 contiguous bytes
//   K, FP4     16 tokens of one kv head, rotated into shared memory and
//              quantised from there by 32-channel items
//   V, FP4     32 token-pair items of the FP4 append
//   Q          one token, 16 rows of head_dim 128 (4 KB in, 4 KB out)
#include "kvq_append.cuh"
#include "kvq_block8.cuh"
#include "kvq_common.cuh"
#include "kvq_host.cuh"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

// warps per CTA (head_dim 256: the FP4 staging buffer keeps within 48 KB)
template <int D>
__host__ __device__ constexpr int rope_warps() { return D == 256 ? 4 : 8; }
constexpr int kQSteps = 4;  // 32-lane steps per query task, all loads in flight together

struct RopeParams {
  kvq_cache c;
  const int32_t* start;
  const int32_t* new_lens;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* table;
  uint16_t* q_out;
  uint16_t* k_out;
  int32_t* flag;
  int64_t q_stride, k_stride, v_stride, table_rows;
  int32_t batch, n_new, hq, rd, interleaved;
  uint32_t blocks;              // 16-token blocks that n_new tokens can touch
  uint32_t pairs;               // token pairs that they can touch
  uint32_t k_tasks, v_tasks, q_tasks;
  uint32_t q_parts;             // query tasks per token
  int32_t early;                // let a dependent launch start at once
};

// New tokens of sequence b: start position and count after every check (0 new
// tokens when the sequence is skipped).
__device__ __forceinline__ int seq_tokens(const RopeParams& p, int b, int64_t& sp) {
  const int32_t s = __ldg(p.start + b);
  int n = p.new_lens ? __ldg(p.new_lens + b) : p.n_new;
  sp = s;
  if (s < 0 || n < 0 || n > p.n_new) {
    if ((threadIdx.x & 31) == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
    return 0;
  }
  if (p.rd > 0 && n > 0 && (int64_t)s + n > p.table_rows) {
    if ((threadIdx.x & 31) == 0) set_flag(p.flag, KVQ_FLAG_POSITION);
    n = (int)max((int64_t)0, p.table_rows - s);
  }
  return n;
}

__device__ __forceinline__ uint32_t bf16x2_from_f32(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Scalar, each step rounded: the packed f32x2 forms of these products and sums
// were seen to give the contracted result on some inputs.
__device__ __forceinline__ void rotate_pair(float x0, float x1, float c, float s, float& y0, float& y1) {
  y0 = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
  y1 = __fadd_rn(__fmul_rn(x1, c), __fmul_rn(x0, s));
}

// The rotation works on items of two 8-channel chunks (a, b) of a row, one
// lane each.  Item j < rd/16 holds 8 whole pairs: the chunks j and j + rd/16
// (pairs (i, i + rd/2)) or 2j and 2j + 1 (pairs (2i, 2i+1)); the items behind
// are the chunks 2j and 2j + 1, passed unchanged.
struct Item {
  uint4 a, b;
};
__device__ __forceinline__ int chunk_a(const RopeParams& p, int j) { return (j < p.rd / 16 && !p.interleaved) ? j : 2 * j; }
__device__ __forceinline__ int chunk_b(const RopeParams& p, int j) {
  return (j < p.rd / 16 && !p.interleaved) ? j + p.rd / 16 : 2 * j + 1;
}

struct Angles {
  float4 c[2], s[2];
};
__device__ __forceinline__ Angles load_angles(const RopeParams& p, int64_t pos, int j) {
  Angles g;
  const float* row = p.table + pos * p.rd + 8 * j;
  g.c[0] = __ldg(reinterpret_cast<const float4*>(row));
  g.c[1] = __ldg(reinterpret_cast<const float4*>(row) + 1);
  g.s[0] = __ldg(reinterpret_cast<const float4*>(row + p.rd / 2));
  g.s[1] = __ldg(reinterpret_cast<const float4*>(row + p.rd / 2) + 1);
  return g;
}

__device__ __forceinline__ void rotate_item(Item& it, const Angles& g, bool interleaved) {
  const float c[8] = {g.c[0].x, g.c[0].y, g.c[0].z, g.c[0].w, g.c[1].x, g.c[1].y, g.c[1].z, g.c[1].w};
  const float s[8] = {g.s[0].x, g.s[0].y, g.s[0].z, g.s[0].w, g.s[1].x, g.s[1].y, g.s[1].z, g.s[1].w};
  uint32_t w[8] = {it.a.x, it.a.y, it.a.z, it.a.w, it.b.x, it.b.y, it.b.z, it.b.w};
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y0, y1;
      rotate_pair(bf16_lo(w[i]), bf16_hi(w[i]), c[i], s[i], y0, y1);
      w[i] = bf16x2_from_f32(y0, y1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0, y1, z0, z1;
      rotate_pair(bf16_lo(w[i]), bf16_lo(w[4 + i]), c[2 * i], s[2 * i], y0, y1);
      rotate_pair(bf16_hi(w[i]), bf16_hi(w[4 + i]), c[2 * i + 1], s[2 * i + 1], z0, z1);
      w[i] = bf16x2_from_f32(y0, z0);
      w[4 + i] = bf16x2_from_f32(y1, z1);
    }
  }
  it.a = make_uint4(w[0], w[1], w[2], w[3]);
  it.b = make_uint4(w[4], w[5], w[6], w[7]);
}

// bf16 bits (no sign) of the largest magnitude of 8 values; >= 0x7F80 when one
// of them is Inf or NaN.
__device__ __forceinline__ uint32_t amax_bits8(const uint4& w) {
  const uint32_t m = bmax_abs(bmax_abs(w.x, w.y), bmax_abs(w.z, w.w));
  return bmax_abs(m, __byte_perm(m, 0u, 0x1032u)) & 0x7FFFu;
}

// The smallest power of two s with amax <= 448 s, from amax's bf16 bits
// (448 = 1.75 * 2^8: the exponent is one higher once the significand passes
// 1.75); 2^-126 at least, 2^120 for Inf and NaN.
__device__ __forceinline__ float block8_scale(uint32_t amax) {
  const int e = (int)(amax >> 7) - 127 - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
  return __uint_as_float((uint32_t)(min(120, max(-126, e)) + 127) << 23);
}

// x / s.  Every scale that an append made is a power of two: then the bf16
// values are multiplied by its exact reciprocal, two at a time (the product is
// exact in bf16 down to 2^-126, where the code is 0).  Any other scale (one
// that the caller wrote) divides in fp32.
struct Quot {
  float s;
  uint32_t inv2;  // the reciprocal as bf16x2, 0: divide
  __device__ explicit Quot(float scale) : s(scale) {
    const uint32_t u = __float_as_uint(scale);
    const bool pow2 = (u & 0x7FFFFFu) == 0u && u >= 0x00800000u && u <= 0x7E800000u;
    inv2 = pow2 ? ((0x7F000000u - u) >> 16) * 0x10001u : 0u;
  }
  // the two values of a word over s
  __device__ __forceinline__ float2 operator()(uint32_t w) const {
    if (inv2 != 0u) {
      uint32_t y;
      asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(y) : "r"(w), "r"(inv2));
      return make_float2(bf16_lo(y), bf16_hi(y));
    }
    return make_float2(__fdiv_rn(bf16_lo(w), s), __fdiv_rn(bf16_hi(w), s));
  }
};

// E4M3 codes (satfinite) of a word's two values: the first in the low byte.
__device__ __forceinline__ uint32_t codes_of_word(uint32_t w, const Quot& q) {
  const float2 y = q(w);
  return e4m3x2_from_f32(y.x, y.y);
}
__device__ __forceinline__ uint2 codes_of_chunk(const uint4& a, const Quot& q) {
  return make_uint2(codes_of_word(a.x, q) | (codes_of_word(a.y, q) << 16), codes_of_word(a.z, q) | (codes_of_word(a.w, q) << 16));
}
// Four kept codes moved to a new scale: r = s_old / s.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float r) {
  const float2 lo = f16x2_to_float2(f16x2_from_e4m3x2(w & 0xFFFFu)), hi = f16x2_to_float2(f16x2_from_e4m3x2(w >> 16));
  return e4m3x2_from_f32(lo.x * r, lo.y * r) | (e4m3x2_from_f32(hi.x * r, hi.y * r) << 16);
}

// ------------------------------------------------------------------ 8-bit tasks
// One 16-token block of one kv head: where it lies, which of its tokens are
// new (bit u) and which are kept.
struct Block8Task {
  uint8_t* grp;
  int64_t first;        // position of the block's token 0
  int64_t row0;         // input row of that token (b * n_new + first - start; may be before the sequence's rows)
  uint32_t fresh, kept;
  int lt;               // the block's first token in its group
  int b, h;
};

// Block r = b * blocks + i of the launch, kv head h.
template <int D>
__device__ __forceinline__ bool block8_task(const RopeParams& p, uint32_t r, int h, Block8Task& t) {
  const uint32_t hkv = (uint32_t)p.c.num_kv_heads;
  t.h = h;
  const int b = (int)(r / p.blocks);
  const uint32_t blk = r - (uint32_t)b * p.blocks;
  int64_t sp;
  const int n = seq_tokens(p, b, sp);
  t.first = 16 * ((sp >> 4) + blk);
  if (n == 0 || t.first >= sp + n) return false;
  const int lo = (int)max((int64_t)0, sp - t.first), hi = (int)min((int64_t)16, sp + n - t.first);
  t.fresh = (0xFFFFu >> (16 - hi)) & (0xFFFFu << lo);
  t.kept = (1u << lo) - 1u;
  t.row0 = (int64_t)b * p.n_new + t.first - sp;
  t.b = b;
  return true;
}

// The block's place in the pool; false when its page is not valid.  Called
// behind the input's loads, so that the page table's latency hides theirs.
template <int D>
__device__ __forceinline__ bool block8_place(const RopeParams& p, Block8Task& t) {
  const int64_t phys = block8_page(p.c, t.b, t.first, p.flag);
  if (phys < 0) return false;
  const Block8Layout L(D, p.c.page_size);
  const int slot = (int)(t.first & (p.c.page_size - 1));
  const int64_t off = block8_group_offset(L, phys, p.c.num_kv_heads, t.h, slot);
  if (!KVQ_IN(off >= 0 && off + L.group_bytes() <= p.c.num_pages * (int64_t)p.c.num_kv_heads * L.page_bytes(), p.flag))
    return false;
  t.grp = static_cast<uint8_t*>(p.c.data) + off;
  t.lt = slot & (L.G - 1);
  return true;
}

// The block's new scale from the warp's amax, with the old one where tokens
// are kept; raise = s_old / s when kept codes have to move (else 1).
__device__ __forceinline__ float block8_new_scale(const Block8Task& t, float old, uint32_t amax, float& raise) {
  float s = block8_scale(amax);
  raise = 1.0f;
  if (t.kept != 0u) {
    if (old >= s)
      s = old;
    else
      raise = __fdiv_rn(fmaxf(old, 0.0f), s);
  }
  return s;
}

// Heads per K group, and warps per group (each 512/D of the block's tokens).
constexpr int kKHeads = 2;
template <int D>
__host__ __device__ constexpr int k8_warps() { return D / 32; }

// `amax` : shared, [k8_warps][kKHeads] of this group; `bar`: its named barrier.
template <int D>
__device__ void append_k8(const RopeParams& p, uint32_t task, uint32_t* amax_s, uint32_t bar) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, W = k8_warps<D>();  // lanes per token, tokens per warp
  static_assert(W * RPS == 16, "a group covers a block");
  const int lane = threadIdx.x & 31, j = lane % LPR, w = (int)(task % W);
  const uint32_t hkv = (uint32_t)p.c.num_kv_heads;
  const uint32_t hgroups = (hkv + kKHeads - 1) / kKHeads;
  const uint32_t g = task / W, r = g / hgroups;
  const int h0 = (int)(g - r * hgroups) * kKHeads;
  const int heads = min(kKHeads, (int)hkv - h0);
  Block8Task t;
  if (!block8_task<D>(p, r, h0, t)) return;  // the whole group
  const Block8Layout L(D, p.c.page_size);
  const int64_t head_bytes = L.page_bytes();  // from one head's group to the next one's
  const int ca = chunk_a(p, j), cb = chunk_b(p, j), u = w * RPS + lane / LPR;
  const bool mine = (t.fresh >> u) & 1u;
  Item it[kKHeads];
  const uint16_t* src = p.k + (t.row0 + u) * p.k_stride + h0 * D;
  const bool turn = mine && j < p.rd / 16;
  Angles ang = {};
  if (turn) ang = load_angles(p, t.first + u, j);
#pragma unroll
  for (int i = 0; i < kKHeads; ++i) {
    it[i].a = it[i].b = make_uint4(0u, 0u, 0u, 0u);
    if (mine && i < heads) {
      it[i].a = __ldg(reinterpret_cast<const uint4*>(src + i * D) + ca);
      it[i].b = __ldg(reinterpret_cast<const uint4*>(src + i * D) + cb);
    }
  }
  const bool ok = block8_place<D>(p, t);
  float old[kKHeads];  // read by every warp before the barrier, written behind it
#pragma unroll
  for (int i = 0; i < kKHeads; ++i)
    old[i] = ok && t.kept != 0u && i < heads ? *reinterpret_cast<const float*>(t.grp + i * head_bytes + L.scale(t.lt >> 4, 0)) : 0.0f;
  uint32_t am[kKHeads];
#pragma unroll
  for (int i = 0; i < kKHeads; ++i) {
    if (turn && i < heads) rotate_item(it[i], ang, p.interleaved);
    if (p.k_out && mine && i < heads) {
      uint4* dst = reinterpret_cast<uint4*>(p.k_out + ((t.row0 + u) * hkv + h0 + i) * D);
      dst[ca] = it[i].a;
      dst[cb] = it[i].b;
    }
    am[i] = __reduce_max_sync(0xFFFFFFFFu, max(amax_bits8(it[i].a), amax_bits8(it[i].b)));
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kKHeads; ++i) amax_s[w * kKHeads + i] = am[i];
  }
  named_barrier_sync(bar, 32 * W);
  if (!ok) return;
#pragma unroll
  for (int i = 0; i < kKHeads; ++i) {
    if (i >= heads) break;
    uint32_t amax = 0u;
#pragma unroll
    for (int k = 0; k < W; ++k) amax = max(amax, amax_s[k * kKHeads + i]);
    if (amax >= 0x7F80u && w == 0 && lane == 0) set_flag(p.flag, KVQ_FLAG_NONFINITE);
    uint8_t* grp = t.grp + i * head_bytes;
    float raise;
    const Quot q(block8_new_scale(t, old[i], amax, raise));
    if (raise != 1.0f) {  // this warp's kept tokens
      const int lo = w * RPS, n = min(RPS, max(0, __popc(t.kept) - lo));
      for (int k = lane; k < n * (D / 16); k += 32) {
        uint4* dst = reinterpret_cast<uint4*>(grp + L.k_code(t.lt + lo + k % n, 16 * (k / n)));
        const uint4 x = *dst;
        *dst = make_uint4(rescale_codes(x.x, raise), rescale_codes(x.y, raise), rescale_codes(x.z, raise),
                          rescale_codes(x.w, raise));
      }
    }
    if (mine) {
      *reinterpret_cast<uint2*>(grp + L.k_code(t.lt + u, 8 * ca)) = codes_of_chunk(it[i].a, q);
      *reinterpret_cast<uint2*>(grp + L.k_code(t.lt + u, 8 * cb)) = codes_of_chunk(it[i].b, q);
    }
    if (w == 0 && lane == 0) *reinterpret_cast<float*>(grp + L.scale(t.lt >> 4, 0)) = q.s;
  }
}

// Bytes of a V row's word w (tokens 2w, 2w+1, 2w+8, 2w+9) whose token is in
// `tokens`.
__device__ __forceinline__ uint32_t v_word_mask(uint32_t tokens, int w) {
  return (((tokens >> (2 * w)) & 1u) ? 0x000000FFu : 0u) | (((tokens >> (2 * w + 1)) & 1u) ? 0x0000FF00u : 0u) |
         (((tokens >> (2 * w + 8)) & 1u) ? 0x00FF0000u : 0u) | (((tokens >> (2 * w + 9)) & 1u) ? 0xFF000000u : 0u);
}

template <int D>
__device__ void append_v8(const RopeParams& p, uint32_t task) {
  constexpr int W = D / 64;  // words (channel pairs) per lane: channels [2 W lane, 2 W (lane + 1))
  const int lane = threadIdx.x & 31;
  Block8Task t;
  const uint32_t hkv = (uint32_t)p.c.num_kv_heads;
  if (!block8_task<D>(p, task / hkv, (int)(task % hkv), t)) return;
  const Block8Layout L(D, p.c.page_size);
  uint32_t x[16][W];
#pragma unroll
  for (int u = 0; u < 16; ++u) {
#pragma unroll
    for (int i = 0; i < W; ++i) x[u][i] = 0u;
    if ((t.fresh >> u) & 1u) {
      const uint16_t* src = p.v + (t.row0 + u) * p.v_stride + t.h * D + 2 * W * lane;
      if constexpr (W == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(src));
        x[u][0] = w.x;
        x[u][1] = w.y;
      } else {
        x[u][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
      }
    }
  }
  if (!block8_place<D>(p, t)) return;
  uint32_t m = 0u;
#pragma unroll
  for (int u = 0; u < 16; ++u)
#pragma unroll
    for (int i = 0; i < W; ++i) m = bmax_abs(m, x[u][i]);
  const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, bmax_abs(m, __byte_perm(m, 0u, 0x1032u)) & 0x7FFFu);
  if (amax >= 0x7F80u && lane == 0) set_flag(p.flag, KVQ_FLAG_NONFINITE);
  float* slot = reinterpret_cast<float*>(t.grp + L.scale(t.lt >> 4, 1));
  float raise;
  const Quot q(block8_new_scale(t, t.kept != 0u ? *slot : 0.0f, amax, raise));
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int u = 0; u < 16; ++u) x[u][i] = codes_of_word(x[u][i], q);  // byte c & 1: channel c of token u
#pragma unroll
  for (int c = 0; c < 2 * W; ++c) {  // channel 2 W lane + c: byte c & 1 of word c / 2
    uint32_t out[4];
    const uint32_t sel = (c & 1) ? 0x5151u : 0x4040u;
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // the tokens 2w, 2w + 1, 2w + 8, 2w + 9
      const uint32_t a = __byte_perm(x[2 * w][c / 2], x[2 * w + 1][c / 2], sel);
      const uint32_t b = __byte_perm(x[2 * w + 8][c / 2], x[2 * w + 9][c / 2], sel);
      out[w] = __byte_perm(a, b, 0x5410u);
    }
    uint4* dst = reinterpret_cast<uint4*>(t.grp + L.v_row(t.lt >> 4, 2 * W * lane + c));
    if (t.fresh != 0xFFFFu) {  // keep the other tokens' bytes
      const uint4 o = *dst;
      const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t mf = v_word_mask(t.fresh, w), mk = v_word_mask(t.kept, w);
        uint32_t old = ow[w];
        if (raise != 1.0f) old = (rescale_codes(old, raise) & mk) | (old & ~mk);
        out[w] = (out[w] & mf) | (old & ~mf);
      }
    }
    *dst = make_uint4(out[0], out[1], out[2], out[3]);
  }
  __syncwarp();
  if (lane == 0) *slot = q.s;
}

// ------------------------------------------------------------------ FP4 tasks
// quantize_plain (kvq_append.cuh) on 16 bf16 values held in registers.
__device__ __noinline__ uint4 quantize_plain_words(uint4 lo, uint4 hi, float S) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  Block16 blk;
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    blk.x[2 * i] = __fdiv_rn(bf16_lo(w[i]), S);
    blk.x[2 * i + 1] = __fdiv_rn(bf16_hi(w[i]), S);
    ok &= isfinite(blk.x[2 * i]) && isfinite(blk.x[2 * i + 1]);
  }
  blk.finite = ok;
  uint32_t sb;
  const uint2 q = quantize_block(blk, sb);
  return make_uint4(q.x, q.y, sb, ok ? 0u : 1u);
}

// Codes and scale byte of one 16-channel K block.
template <bool NV>
__device__ __forceinline__ uint2 quantize_k_block(uint4 lo, uint4 hi, float S, uint32_t& sb, int32_t* flag) {
  Raw16 kb;
  kb.w[0] = lo.x; kb.w[1] = lo.y; kb.w[2] = lo.z; kb.w[3] = lo.w;
  kb.w[4] = hi.x; kb.w[5] = hi.y; kb.w[6] = hi.z; kb.w[7] = hi.w;
  const uint32_t a = block_amax_bits(kb.w);
  kb.amax = __uint_as_float(a << 16);
  kb.finite = a < 0x7F80u;
  if constexpr (NV) {
    float y[16];
    if (nv_fast_scale(S) && nv_quotients(kb, S, __frcp_rn(S), y, sb)) {
      const float s = e4m3_to_f32(sb);
      return k_codes_f32(y, s, __frcp_rn(s));
    }
  } else if (kb.finite) {
    sb = block_scale_byte(kb.amax);
    const float s = e4m3_to_f32(sb);
    return k_codes_finite(kb.w, s, scale_recip(s));
  }
  const uint4 r = quantize_plain_words(lo, hi, S);
  if (r.w) set_flag(flag, KVQ_FLAG_NONFINITE);
  sb = r.z;
  return make_uint2(r.x, r.y);
}

// 16 tokens (from `tile` of the sequence's new tokens) of one kv head.
template <int D, bool NV>
__device__ void append_k4(const RopeParams& p, uint32_t task, uint4* stage) {
  constexpr int LPR = D / 16, RPS = 32 / LPR;
  const int lane = threadIdx.x & 31, j = lane % LPR;
  const uint32_t hkv = (uint32_t)p.c.num_kv_heads;
  const uint32_t r = task / hkv;
  const int h = (int)(task - r * hkv);
  const int b = (int)(r / p.blocks);
  const int t0 = 16 * (int)(r - (uint32_t)b * p.blocks);
  int64_t sp;
  const int n = min(16, seq_tokens(p, b, sp) - t0);
  if (n <= 0) return;
  const int64_t row0 = (int64_t)b * p.n_new + t0;
  const int ca = chunk_a(p, j), cb = chunk_b(p, j);
#pragma unroll 4
  for (int u = lane / LPR; u < n; u += RPS) {
    const uint4* src = reinterpret_cast<const uint4*>(p.k + (row0 + u) * p.k_stride + h * D);
    Item it;
    it.a = __ldg(src + ca);
    it.b = __ldg(src + cb);
    if (j < p.rd / 16) rotate_item(it, load_angles(p, sp + t0 + u, j), p.interleaved);
    if (p.k_out) {
      uint4* dst = reinterpret_cast<uint4*>(p.k_out + ((row0 + u) * hkv + h) * D);
      dst[ca] = it.a;
      dst[cb] = it.b;
    }
    stage[u * (D / 8) + ca] = it.a;
    stage[u * (D / 8) + cb] = it.b;
  }
  __syncwarp();
  const float S = NV ? __ldg(static_cast<const float*>(p.c.k_scale) + h) : 1.0f;
  const int G = p.c.page_size < 128 ? p.c.page_size : 128;
  for (int i = lane; i < n * (D / 32); i += 32) {  // 32 channels of one token
    const int u = i / (D / 32), c32 = i % (D / 32);
    const uint4* w = stage + u * (D / 8) + 4 * c32;
    int ls = 0;
    uint8_t* grp = fp4_group<D>(p.c, b, sp + t0 + u, h, ls, p.flag);
    if (grp == nullptr) continue;
    uint32_t s0, s1;
    const uint2 c0 = quantize_k_block<NV>(w[0], w[1], S, s0, p.flag);
    const uint2 c1 = quantize_k_block<NV>(w[2], w[3], S, s1, p.flag);
    *reinterpret_cast<uint4*>(grp + ls * (D / 2) + 16 * c32) = make_uint4(c0.x, c0.y, c1.x, c1.y);
    *reinterpret_cast<uint16_t*>(grp + G * (D / 2) + ls * (D / 16) + 2 * c32) = (uint16_t)(s0 | (s1 << 8));
  }
}

// 32 token-pair items of 16 channels (the FP4 append's V items).
template <int D, bool NV>
__device__ void append_v4(const RopeParams& p, uint32_t task) {
  constexpr int NB = D / 16;
  const uint32_t hkv = (uint32_t)p.c.num_kv_heads;
  const uint32_t item = task * 32u + (threadIdx.x & 31);
  const int j0 = (int)(item % NB);
  const uint32_t r = item / NB;
  const uint32_t r2 = r / hkv;
  const int h = (int)(r - r2 * hkv);
  const int b = (int)(r2 / p.pairs);
  if (b >= p.batch) return;
  int64_t sp;
  const int n = seq_tokens(p, b, sp);
  const int64_t pos = 2 * ((sp >> 1) + (r2 - (uint32_t)b * p.pairs)), end = sp + n;
  if (n == 0 || pos >= end) return;
  int ls = 0;
  uint8_t* grp = fp4_group<D>(p.c, b, pos, h, ls, p.flag);
  if (grp == nullptr) return;
  const bool mine0 = pos >= sp, mine1 = pos + 1 < end;
  const uint16_t* src0 = p.v + ((int64_t)b * p.n_new + (pos - sp)) * p.v_stride + h * D + 16 * j0;
  append_v_item<D, NV>(p.c, grp, ls, h, j0, mine0, mine1, src0, src0 + p.v_stride, p.flag);
}

// ------------------------------------------------------------------ queries
template <int D>
__device__ void rotate_q(const RopeParams& p, uint32_t task) {
  constexpr int LPR = D / 16, RPS = 32 / LPR;
  const int lane = threadIdx.x & 31, j = lane % LPR;
  const uint32_t tok = task / p.q_parts;
  const int h0 = (int)(task - tok * p.q_parts) * kQSteps * RPS + lane / LPR;
  const int b = (int)(tok / (uint32_t)p.n_new);
  const int t = (int)(tok - (uint32_t)b * p.n_new);
  int64_t sp;
  if (t >= seq_tokens(p, b, sp)) return;
  const int ca = chunk_a(p, j), cb = chunk_b(p, j);
  const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)tok * p.q_stride);
  uint4* dst = reinterpret_cast<uint4*>(p.q_out + (int64_t)tok * p.hq * D);
  const bool turn = j < p.rd / 16;
  Angles g = {};
  if (turn) g = load_angles(p, sp + t, j);
  Item it[kQSteps];
#pragma unroll
  for (int i = 0; i < kQSteps; ++i) {
    const int h = h0 + i * RPS;
    if (h < p.hq) {
      it[i].a = __ldg(src + h * (D / 8) + ca);
      it[i].b = __ldg(src + h * (D / 8) + cb);
    }
  }
#pragma unroll
  for (int i = 0; i < kQSteps; ++i) {
    const int h = h0 + i * RPS;
    if (h >= p.hq) break;
    if (turn) rotate_item(it[i], g, p.interleaved);
    dst[h * (D / 8) + ca] = it[i].a;
    dst[h * (D / 8) + cb] = it[i].b;
  }
}

// FORMAT: KVQ_FORMAT_*.  Tasks in the order K, V, Q.
template <int D, int FORMAT>
__global__ void __launch_bounds__(32 * rope_warps<D>(), 4) rope_append_kernel(const RopeParams p) {
  constexpr bool kFp4 = FORMAT != KVQ_FORMAT_FP8_E4M3_BLOCK;
  __shared__ uint4 stage[kFp4 ? rope_warps<D>() * 16 * (D / 8) : 1];
  __shared__ uint32_t amax_s[rope_warps<D>() * kKHeads];
  if (p.early) grid_launch_dependents();
  const int warp = threadIdx.x >> 5;
  uint32_t task = blockIdx.x * rope_warps<D>() + warp;
  if (task < p.k_tasks) {
    if constexpr (kFp4)
      append_k4<D, FORMAT == KVQ_FORMAT_NVFP4>(p, task, stage + warp * 16 * (D / 8));
    else  // the group's warps lie in one CTA
      append_k8<D>(p, task, amax_s + warp / k8_warps<D>() * k8_warps<D>() * kKHeads, 1 + warp / k8_warps<D>());
    return;
  }
  task -= p.k_tasks;
  if (task < p.v_tasks) {
    if constexpr (kFp4)
      append_v4<D, FORMAT == KVQ_FORMAT_NVFP4>(p, task);
    else
      append_v8<D>(p, task);
    return;
  }
  task -= p.v_tasks;
  if (task < p.q_tasks) rotate_q<D>(p, task);
}

__global__ void __launch_bounds__(256) rope_table_kernel(int64_t n, int32_t half, double base, float* table) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n * half) return;
  const int64_t pos = i / half;
  const int f = (int)(i % half);
  double s, c;
  sincos((double)pos * pow(base, -(double)f / (double)half), &s, &c);
  table[pos * 2 * half + f] = (float)c;
  table[pos * 2 * half + half + f] = (float)s;
}

template <int D>
void launch_rope(RopeParams p, cudaStream_t s) {
  constexpr int kThreads = 32 * rope_warps<D>();
  const int64_t tasks = (int64_t)p.k_tasks + p.v_tasks + p.q_tasks;
  const unsigned grid = (unsigned)((tasks + rope_warps<D>() - 1) / rope_warps<D>());
  // A decode step's append is over in one wave: a dependent launch may take
  // its SM slots at once.  A longer one would have them occupied by CTAs that
  // only wait.
  p.early = (int64_t)grid <= 2 * (int64_t)device_sm_count() ? 1 : 0;
  switch (p.c.format) {
    case KVQ_FORMAT_FP4_E2M1_E4M3_G16:
      rope_append_kernel<D, KVQ_FORMAT_FP4_E2M1_E4M3_G16><<<grid, kThreads, 0, s>>>(p);
      break;
    case KVQ_FORMAT_NVFP4: rope_append_kernel<D, KVQ_FORMAT_NVFP4><<<grid, kThreads, 0, s>>>(p); break;
    default:
      if constexpr (D != 256) rope_append_kernel<D, KVQ_FORMAT_FP8_E4M3_BLOCK><<<grid, kThreads, 0, s>>>(p);
      break;
  }
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_rope_table(int64_t num_positions, int32_t rotary_dim, double base, float* table,
                                     kvq_stream stream) {
  if (num_positions < 0 || rotary_dim < 2 || rotary_dim > 512 || (rotary_dim & 1) || !(base > 0.0) || !(base < 1e300))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_positions == 0) return KVQ_OK;
  if (table == nullptr || !aligned_to(table, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_positions > ((int64_t)1 << 31)) return KVQ_ERR_UNSUPPORTED;
  const int32_t half = rotary_dim / 2;
  const int64_t ctas = (num_positions * half + 255) / 256;
  if (ctas > 0x7FFFFFFF) return KVQ_ERR_UNSUPPORTED;
  rope_table_kernel<<<(unsigned)ctas, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(num_positions, half, base, table);
  return launch_status();
}

extern "C" kvq_status kvq_rope_append(const kvq_cache* cache, int32_t batch, int32_t n_new, const int32_t* d_start_pos,
                                      const int32_t* d_new_lens, int32_t num_q_heads, const void* q, int64_t q_stride,
                                      const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                      const float* table, int64_t table_rows, int32_t rotary_dim, int32_t interleaved,
                                      void* q_out, void* k_out, int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 0 || n_new < 0 || num_q_heads < 0 || cache == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if (cache->format == KVQ_FORMAT_FP8_E4M3_HEAD) return KVQ_ERR_UNSUPPORTED;
  const bool fp8 = cache->format == KVQ_FORMAT_FP8_E4M3_BLOCK;
  const kvq_status st = fp8 ? check_block8_cache(cache, batch) : check_cache(cache, batch);
  if (st != KVQ_OK) return st;
  const int32_t D = cache->head_dim, hkv = cache->num_kv_heads;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0 || (interleaved != 0 && interleaved != 1))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (rotary_dim > 0 && (table == nullptr || !aligned_to(table, 16) || table_rows < 0)) return KVQ_ERR_INVALID_ARGUMENT;
  if (batch == 0 || n_new == 0) return KVQ_OK;
  if (d_start_pos == nullptr || k == nullptr || v == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads > 0 && (q == nullptr || q_out == nullptr)) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads == 0 && (q != nullptr || q_out != nullptr)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(q_out, 16) || !aligned_to(k_out, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < (int64_t)hkv * D || v_stride < (int64_t)hkv * D)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads > 0 && (q_stride % 8 != 0 || q_stride < (int64_t)num_q_heads * D)) return KVQ_ERR_INVALID_ARGUMENT;
  if (q_out == q && num_q_heads > 0 && q_stride != (int64_t)num_q_heads * D) return KVQ_ERR_INVALID_ARGUMENT;
  if (k_out == k && k_stride != (int64_t)hkv * D) return KVQ_ERR_INVALID_ARGUMENT;

  RopeParams p = {};
  p.c = *cache;
  p.start = d_start_pos;
  p.new_lens = d_new_lens;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.table = table;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.flag = d_err_flag;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.table_rows = table_rows;
  p.batch = batch;
  p.n_new = n_new;
  p.hq = num_q_heads;
  p.rd = rotary_dim;
  p.interleaved = interleaved;
  // 16-token blocks aligned to positions can be cut at both ends (8 bit);
  // the FP4 K tasks count from the first new token
  p.blocks = fp8 ? (uint32_t)(((int64_t)n_new + 30) / 16) : (uint32_t)(((int64_t)n_new + 15) / 16);
  p.pairs = (uint32_t)(n_new / 2 + 1);
  const int64_t rows_per_q = (int64_t)kQSteps * 32 / (D / 16);
  p.q_parts = (uint32_t)((num_q_heads + rows_per_q - 1) / rows_per_q);
  const double limit = (double)(1 << 30);  // 32-bit task and item indices
  const double vt = (double)batch * p.blocks * hkv;
  const double kt = fp8 ? (double)batch * p.blocks * ((hkv + kKHeads - 1) / kKHeads) * (D / 32) : vt, qt = (double)batch * n_new * p.q_parts;
  const double vi = (double)batch * p.pairs * hkv * (D / 16);
  if (kt > limit || vt > limit || qt > limit || vi > limit) return KVQ_ERR_UNSUPPORTED;
  p.k_tasks = (uint32_t)kt;
  p.v_tasks = fp8 ? (uint32_t)vt : ((uint32_t)vi + 31u) / 32u;
  p.q_tasks = (uint32_t)qt;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 64)
    launch_rope<64>(p, s);
  else if (D == 128)
    launch_rope<128>(p, s);
  else
    launch_rope<256>(p, s);
  return launch_status();
}

extern "C" kvq_status kvq_fp8_block_append(const kvq_cache* cache, int32_t batch, int32_t n_new,
                                           const int32_t* d_start_pos, const int32_t* d_new_lens, const void* k,
                                           const void* v, int32_t* d_err_flag, kvq_stream stream) {
  if (cache == nullptr || cache->format != KVQ_FORMAT_FP8_E4M3_BLOCK) return KVQ_ERR_INVALID_ARGUMENT;
  const int64_t stride = (int64_t)cache->num_kv_heads * cache->head_dim;
  return kvq_rope_append(cache, batch, n_new, d_start_pos, d_new_lens, 0, nullptr, 0, k, stride, v, stride, nullptr, 0,
                         0, 0, nullptr, nullptr, d_err_flag, stream);
}

extern "C" size_t kvq_fp8_block_pool_bytes(int64_t num_pages, int32_t num_kv_heads, int32_t page_size,
                                           int32_t head_dim) {
  if (num_pages < 0 || num_kv_heads < 1 || !is_pow2_page(page_size) || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)num_pages * (size_t)num_kv_heads * (size_t)Block8Layout(head_dim, page_size).page_bytes();
}
