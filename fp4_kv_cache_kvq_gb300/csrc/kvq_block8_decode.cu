// kvq_block8_decode.cu -- split-K flash-decode attention over the 8-bit block
// cache (one query token per sequence), and its C entry point.
//
// Mathematics.  For one (sequence, kv head) unit with G query rows,
//   S_t = q . code_t,  y_t = S_t * (softmax_scale log2 e * sK[t / 16]),
//   o = sum_t 2^(y_t - m) sV[t / 16] code_t / sum_t 2^(y_t - m)
// in one pass, with a running maximum m (raised only when a score passes it
// by more than 8) and fp32 sums.  The scales are constant over a 16-token
// slice, which is the M of one mma.m16n8k16 product for S and the K of one
// for o: so codes enter the products as they are (E4M3 -> f16 is exact), and
// a slice costs one multiply per score for sK and one FMA per accumulator for
// sV, which also folds the slice's sum into o.  q is scaled by a power of two
// per head, so its bf16 values are exact in f16 down to 2^-31 of the row's largest; p = 2^(y - m) is rounded to
// f16 (2^-11 relative) for the second product.
//
// What bounds it: HBM, 2 Hkv (d + 1/4) bytes a position against 4 Hq d flop.
// Work split: all units' chunks (64 tokens, 128 at head_dim 64) laid end to end and cut into equal
// ranges, one per CTA of a persistent grid, so ragged lengths balance to
// within a chunk; a CTA leaves one partial (m, l, o) per unit it touches and
// the merge (kvq_merge.cu) joins them.
// CTA: 4 consumer warps, a quarter of a chunk each, and a producer warp that
// keeps a ring of stages full with one bulk copy per group (mbarriers; every
// wait bounded).
#include "kvq_block8.cuh"
#include "kvq_common.cuh"
#include "kvq_decode.cuh"
#include "kvq_host.cuh"

namespace kvq {
namespace {

constexpr int kB8Warps = 4;    // consumer warps
// Tokens per stage: 16 KB of codes at either head size (at head_dim 64 a stage
// of 64 tokens left too little to do between two hand-offs).
template <int D>
__host__ __device__ constexpr int chunk8() { return D == 64 ? 128 : 64; }
constexpr int kB8Threads = 32 * (kB8Warps + 1);
// CTAs per SM and stages per CTA.  head_dim 128: two CTAs of four stages, whose
// 146 registers spill nothing, run medium batches in 49.0 us against 50.2 for
// three of three stages (16 x 8192 positions, 8 kv and 64 query heads) and long
// ones alike (32 x 32768: 311.7 us); head_dim 64: three of three, 85 against
// 88 us (16 x 32768).
template <int D>
__host__ __device__ constexpr int ctas8() { return D == 128 ? 2 : 3; }
template <int D>
__host__ __device__ constexpr int stages8() { return D == 128 ? 4 : 3; }

struct Decode8Params {
  const int32_t* lens;
  kvq_cache c;
  const uint16_t* q;
  float* part_o;
  float* part_ml;
  int2* unit_rec;
  int32_t* flag;
  int32_t batch, hkv, g, hq, window;  // window: 0 (the shared walk's parameter)
  float qk_log2;                      // softmax_scale * log2(e)
  int64_t n_slots;
  void* out;                          // direct: the result, else nullptr
  int32_t out_bf16;
  uint64_t wait_ns;                   // a test's limit of the work waits, or 0
};

// Positions of sequence b: no more than its pages can hold (a longer length is
// flagged where its last chunk is read).
__device__ __forceinline__ int32_t walk_len(const Decode8Params& p, int b) {
  return (int32_t)min((int64_t)__ldg(p.lens + b), (int64_t)p.c.max_pages_per_seq * p.c.page_size);
}

// A consumer's wait for a stage to land and the producer's for a free one: the
// library's limit or, in the instantiation for tests, theirs.
template <bool TEST>
__device__ __forceinline__ bool work_wait8(const Decode8Params& p, uint32_t bar, uint32_t parity) {
  if constexpr (TEST)
    return mbar_wait_limit(bar, parity, p.wait_ns);
  else
    return mbar_wait(bar, parity);
}

// Compile-time view of one group of GT tokens (see Block8Layout).
template <int D, int GT>
struct Grp8 {
  static constexpr int kV = GT * D;
  static constexpr int kScales = 2 * GT * D;
  static constexpr int kBytes = 2 * GT * D + (GT >= 32 ? GT / 2 : 16);
  static constexpr int kCopies = chunk8<D>() / GT;  // groups per stage
};

template <int D>
struct Geo8 {
  static constexpr int kSlices = chunk8<D>() / (16 * kB8Warps);  // 16-token slices per warp
  static constexpr int kStageBytes =
      (chunk8<D>() / 16 * Grp8<D, 16>::kBytes + 127) / 128 * 128;  // the largest of the group sizes
  static constexpr int kFlushBytes = kB8Warps * kNG * (D + 2) * 4;
  static constexpr int kSmemBytes = stages8<D>() * kStageBytes + kFlushBytes + 2 * stages8<D>() * 8 + 2 * stages8<D>() * 4 + 16 + 128;
};

template <int D>
struct Smem8 {
  uint8_t* stages;
  float* flush_o;   // [warp][row][D]
  float* flush_m;   // [warp][row]
  float* flush_l;   // [warp][row]
  uint64_t* full;
  uint64_t* empty;
  int* ntok;
  uint32_t* good;   // bit i: slice i of the stage lies in a valid page
  int* abort;
};

template <int D>
__device__ __forceinline__ Smem8<D> carve8(uint8_t* raw) {
  using G = Geo8<D>;
  Smem8<D> s;
  uint8_t* ptr = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
  s.stages = ptr;
  ptr += stages8<D>() * G::kStageBytes;
  s.flush_o = reinterpret_cast<float*>(ptr);
  ptr += kB8Warps * kNG * D * 4;
  s.flush_m = reinterpret_cast<float*>(ptr);
  ptr += kB8Warps * kNG * 4;
  s.flush_l = reinterpret_cast<float*>(ptr);
  ptr += kB8Warps * kNG * 4;
  s.full = reinterpret_cast<uint64_t*>(ptr);
  ptr += stages8<D>() * 8;
  s.empty = reinterpret_cast<uint64_t*>(ptr);
  ptr += stages8<D>() * 8;
  s.ntok = reinterpret_cast<int*>(ptr);
  ptr += stages8<D>() * 4;
  s.good = reinterpret_cast<uint32_t*>(ptr);
  ptr += stages8<D>() * 4;
  s.abort = reinterpret_cast<int*>(ptr);
  return s;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Four E4M3 codes of a word -> two f16x2 (bytes 0, 1 and bytes 2, 3).
__device__ __forceinline__ void f16x2x2_from_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// ------------------------------------------------------------------ producer
// The producer warp.  Lane i < kCopies issues the copy of the stage's group i.
// The page table's entries come 32 at a time into the lanes' registers, the
// next 32 ahead of their use, so that no copy waits for a lookup (a lookup per
// copy bound the pages of 16 tokens to 0.78 of the rate).  Tokens of a group
// whose page is not valid are left out: its slices lose their bit.
template <int D, int GT, bool TEST>
__device__ void producer8(const Decode8Params& p, Smem8<D>& sm, Walker wk, int64_t v1) {
  using R = Grp8<D, GT>;
  constexpr int C = chunk8<D>();
  const int lane = threadIdx.x & 31;
  const int P = p.c.page_size, lg_p = __ffs(P) - 1;
  const int64_t page_bytes = (int64_t)(P / GT) * R::kBytes;
  const uint8_t* pool = static_cast<const uint8_t*>(p.c.data);
  const auto entry = [&](int b, int64_t pg) -> int64_t {
    if (pg >= p.c.max_pages_per_seq) return -1;
    const int64_t at = (int64_t)b * p.c.max_pages_per_seq + pg;
    return p.c.page_table ? (int64_t)__ldg(p.c.page_table + at) : at;
  };
  int wb = -1;              // the window of 32 entries held: sequence and first page
  int64_t w0 = 0, win = -1, nxt = -1;
  uint32_t it = 0;
  for (; wk.v < v1; advance<C>(p, wk), ++it) {
    const uint32_t s = it % stages8<D>();
    const int64_t tok0 = (int64_t)wk.c * C;
    const int ntok = (int)min((int64_t)C, walk_len(p, wk.b) - tok0);
    if (wk.c == wk.nch - 1 && lane == 0 && __ldg(p.lens + wk.b) > walk_len(p, wk.b)) set_flag(p.flag, KVQ_FLAG_PAGE_OOB);
    const int64_t pg0 = tok0 >> lg_p, pg1 = (tok0 + ntok - 1) >> lg_p;
    if (wk.b != wb || pg0 < w0 || pg1 >= w0 + 32) {
      if (wk.b == wb && pg0 == w0 + 32) {
        win = nxt;
      } else {
        win = entry(wk.b, pg0 + lane);
      }
      wb = wk.b;
      w0 = pg0;
      nxt = entry(wb, w0 + 32 + lane);
    }
    const int64_t pos = tok0 + lane * GT;
    const bool need = lane < R::kCopies && lane * GT < ntok;
    const int64_t phys = __shfl_sync(0xFFFFFFFFu, win, need ? (int)((pos >> lg_p) - w0) : 0);
    const int64_t src = (phys * p.hkv + wk.h) * page_bytes + ((int)(pos & (P - 1)) / GT) * R::kBytes;
    bool ok = need && phys >= 0 && phys < p.c.num_pages;
    if (need && !ok) set_flag(p.flag, KVQ_FLAG_PAGE_OOB);
    ok = ok && KVQ_IN(src >= 0 && src + R::kBytes <= p.c.num_pages * (int64_t)p.hkv * page_bytes &&
                          (lane + 1) * R::kBytes <= Geo8<D>::kStageBytes,
                      p.flag);
    const uint32_t got = __ballot_sync(0xFFFFFFFFu, ok);
    bool live = true;
    if (it >= (uint32_t)stages8<D>() && !work_wait8<TEST>(p, smem_addr(&sm.empty[s]), ((it / stages8<D>()) + 1) & 1)) {
      set_flag(p.flag, KVQ_FLAG_TIMEOUT);
      *reinterpret_cast<volatile int*>(sm.abort) = 1;
      live = false;
    }
    if (!__all_sync(0xFFFFFFFFu, live && *reinterpret_cast<volatile int*>(sm.abort) == 0)) break;
    const uint32_t full = smem_addr(&sm.full[s]);
    if (lane == 0) {
      uint32_t good = 0;
#pragma unroll
      for (int i = 0; i < R::kCopies; ++i)
        if ((got >> i) & 1u) good |= ((1u << (GT / 16)) - 1u) << (i * (GT / 16));
      sm.ntok[s] = ntok;
      sm.good[s] = good;
      mbar_arrive_expect_tx(full, (uint32_t)__popc(got) * R::kBytes);
    }
    __syncwarp();
    if (ok) bulk_g2s(smem_addr(sm.stages) + s * Geo8<D>::kStageBytes + lane * R::kBytes, pool + src, R::kBytes, full);
  }
  // every copy still in flight lands before the CTA can retire
  for (uint32_t j = it > (uint32_t)stages8<D>() ? it - stages8<D>() : 0; j < it; ++j) {
    if (!mbar_wait(smem_addr(&sm.full[j % stages8<D>()]), (j / stages8<D>()) & 1)) {
      set_flag(p.flag, KVQ_FLAG_TIMEOUT);
      break;
    }
  }
}

// ------------------------------------------------------------------ consumers
template <int D>
struct State8 {
  float o[D / 16][4];   // channel 16 mt + g (+8), query rows 2t, 2t + 1
  uint32_t qf[D / 8];   // B fragments: channels 16 i + 4t .. + 3 of query row g
  float cs[2], m[2], l[2];
};

// A unit's query rows, loaded ahead of the last unit's flush (which hides them).
template <int D>
__device__ __forceinline__ void load_rows8(const Decode8Params& p, uint2 (&w)[D / 16], int b, int h) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t qrow = (int64_t)b * p.hq + (int64_t)h * p.g + g;
  const bool row = g < p.g && KVQ_IN(qrow < (int64_t)p.batch * p.hq, p.flag);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    w[i] = row ? __ldcg(reinterpret_cast<const uint2*>(p.q + qrow * D + 16 * i + 4 * t)) : make_uint2(0u, 0u);
}

template <int D>
__device__ __forceinline__ void begin_unit8(const Decode8Params& p, State8<D>& st, const uint2 (&w)[D / 16]) {
  const int lane = threadIdx.x & 31, t = lane & 3;
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    amax = max(amax, max(max((w[i].x << 16) & 0x7FFF0000u, w[i].x & 0x7FFF0000u),
                         max((w[i].y << 16) & 0x7FFF0000u, w[i].y & 0x7FFF0000u)));
  }
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  // power-of-two prescale: max |q| * 2^k in [2^14, 2^15) keeps bf16 values exact in f16
  // from 2^-17 up (f16's smallest step is 2^-24)
  int k = 0;
  if (amax > 0u && amax < 0x7F800000u) k = min(100, max(-113, 14 - ((int)(amax >> 23) - 127)));
  const float up = __uint_as_float((uint32_t)(k + 127) << 23);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    st.qf[2 * i] = pack_f16x2(bf16_lo(w[i].x) * up, bf16_hi(w[i].x) * up);
    st.qf[2 * i + 1] = pack_f16x2(bf16_lo(w[i].y) * up, bf16_hi(w[i].y) * up);
  }
  // the factor, exactly undone in the score scale; a query with Inf or NaN makes
  // its row NaN (the finite maximum keeps the row from counting as empty)
  const float back = amax < 0x7F800000u ? __uint_as_float((uint32_t)(127 - k) << 23) : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float f = __shfl_sync(0xFFFFFFFFu, back, (2 * t + i) * 4);
    st.cs[i] = p.qk_log2 * f;
    st.m[i] = f == f ? -INFINITY : 0.0f;
    st.l[i] = 0.0f;
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) st.o[mt][i] = 0.0f;
}

// Slice `sl` of a stage (16 tokens).  PARTIAL: only tokens [0, ntok) of it are
// attended (the last chunk of a unit).  LAST: the warp is done with the stage
// once the V codes are in registers.
template <int D, int GT, bool PARTIAL, bool LAST>
__device__ __forceinline__ void consume8(State8<D>& st, uint32_t stage, int sl, int ntok, uint32_t empty_bar) {
  using R = Grp8<D, GT>;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t grp = stage + (uint32_t)((16 * sl / GT) * R::kBytes);
  const int blk = (16 * sl % GT) / 16;  // the slice's block in its group
  const uint2 sc = lds64(grp + R::kScales + 8 * blk);
  const float ks = __uint_as_float(sc.x), vs = __uint_as_float(sc.y);

  // S^T = K Q^T: 16 tokens x 16 channels per step; matrices (tokens 0-7,
  // 8-15) x (channel block, the next one).  Two chains of products, as one of
  // eight in a row is the longest wait of a slice (16 x 8192: 48.45 -> 48.15 us, three
  // runs of each in turn, whose medians differ by 0.05)
  float S[4] = {0.f, 0.f, 0.f, 0.f}, S2[4] = {0.f, 0.f, 0.f, 0.f};
  const uint32_t ka = grp + (uint32_t)((2 * blk + ((lane >> 3) & 1)) * 8 * D + (lane >> 4) * 128 + (lane & 7) * 16);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t r[4], a[8];
    ldmatrix_x4(ka + 256 * i, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) f16x2x2_from_e4m3x4(r[j], a[2 * j], a[2 * j + 1]);
    mma_f16_16816(S, a[0], a[2], a[1], a[3], st.qf[4 * i], st.qf[4 * i + 1]);
    mma_f16_16816(S2, a[4], a[6], a[5], a[7], st.qf[4 * i + 2], st.qf[4 * i + 3]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) S[i] += S2[i];
  const float c0 = st.cs[0] * ks, c1 = st.cs[1] * ks;
  float y0 = S[0] * c0, y1 = S[1] * c1, y2 = S[2] * c0, y3 = S[3] * c1;
  if (PARTIAL) {
    if (g >= ntok) y0 = y1 = -INFINITY;
    if (g + 8 >= ntok) y2 = y3 = -INFINITY;
  }
  float m0 = fmaxf(y0, y2), m1 = fmaxf(y1, y3);
  float al0 = 1.0f, al1 = 1.0f;
  const bool rescale = __any_sync(0xFFFFFFFFu, m0 > st.m[0] + kLazySlack || m1 > st.m[1] + kLazySlack);
  if (rescale) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, o));
      m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, o));
    }
    const float n0 = fmaxf(st.m[0], m0), n1 = fmaxf(st.m[1], m1);
    al0 = (st.m[0] == -INFINITY) ? 0.0f : fast_exp2(st.m[0] - n0);
    al1 = (st.m[1] == -INFINITY) ? 0.0f : fast_exp2(st.m[1] - n1);
    st.l[0] *= al0;
    st.l[1] *= al1;
    st.m[0] = n0;
    st.m[1] = n1;
  }
  const float r0 = st.m[0] == -INFINITY ? 0.0f : st.m[0], r1 = st.m[1] == -INFINITY ? 0.0f : st.m[1];
  const float p0 = fast_exp2(y0 - r0), p1 = fast_exp2(y1 - r1), p2 = fast_exp2(y2 - r0), p3 = fast_exp2(y3 - r1);
  st.l[0] += p0 + p2;
  st.l[1] += p1 + p3;
  const uint32_t pa = movmatrix_trans(pack_f16x2(p0, p1)), pb = movmatrix_trans(pack_f16x2(p2, p3));

  // O^T += sV (V^T P^T): matrices = 8 channels x the slice's 16 tokens; a word
  // holds this thread's tokens 2t, 2t+1, 2t+8, 2t+9
  uint32_t v[D / 8];
  const uint32_t va = grp + (uint32_t)(R::kV + (blk * D + lane) * 16);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t r[4];
    ldmatrix_x4(va + 512 * i, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = r[j];
  }
  if (LAST) mbar_arrive(empty_bar);
  if (PARTIAL) {  // stale bytes of tokens behind the end must not inject NaN
    const uint32_t keep = (2 * t < ntok ? 0x000000FFu : 0u) | (2 * t + 1 < ntok ? 0x0000FF00u : 0u) |
                          (2 * t + 8 < ntok ? 0x00FF0000u : 0u) | (2 * t + 9 < ntok ? 0xFF000000u : 0u);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) v[i] &= keep;
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    uint32_t a0, a1, a2, a3;
    f16x2x2_from_e4m3x4(v[2 * mt], a0, a2);
    f16x2x2_from_e4m3x4(v[2 * mt + 1], a1, a3);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    mma_f16_16816(acc, a0, a1, a2, a3, pa, pb);
    if (rescale) {
      st.o[mt][0] *= al0;
      st.o[mt][1] *= al1;
      st.o[mt][2] *= al0;
      st.o[mt][3] *= al1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) st.o[mt][i] = fmaf(acc[i], vs, st.o[mt][i]);
  }
}

__device__ __forceinline__ void store_out8(const Decode8Params& p, int64_t row, int d, int c4, float4 o) {
  if (p.out_bf16) {
    uint2 v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(v.x) : "f"(o.y), "f"(o.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(v.y) : "f"(o.w), "f"(o.z));
    *(reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * d) + c4) = v;
  } else {
    *(reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * d) + c4) = o;
  }
}

// Combine the four warps' states for one unit and write the CTA's partial into
// slot `slot` (DIRECT: the result, to the output rows from `slot` on).
template <int D, bool DIRECT>
__device__ void flush_unit8(const Decode8Params& p, State8<D>& st, Smem8<D>& sm, int64_t slot) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    st.l[0] += __shfl_xor_sync(0xFFFFFFFFu, st.l[0], o);
    st.l[1] += __shfl_xor_sync(0xFFFFFFFFu, st.l[1], o);
  }
  // scores that were all NaN raised no maximum: a finite one keeps their NaN sums
  // from counting as empty
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (st.l[i] != st.l[i] && st.m[i] == -INFINITY) st.m[i] = 0.0f;
  named_barrier_sync(1, 32 * kB8Warps);  // the previous flush has been read
  float* ow = sm.flush_o + warp * kNG * D;
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    const int c0 = 16 * mt + g;
    ow[(2 * t) * D + c0] = st.o[mt][0];
    ow[(2 * t + 1) * D + c0] = st.o[mt][1];
    ow[(2 * t) * D + c0 + 8] = st.o[mt][2];
    ow[(2 * t + 1) * D + c0 + 8] = st.o[mt][3];
  }
  if (g == 0) {
    sm.flush_m[warp * kNG + 2 * t] = st.m[0];
    sm.flush_m[warp * kNG + 2 * t + 1] = st.m[1];
    sm.flush_l[warp * kNG + 2 * t] = st.l[0];
    sm.flush_l[warp * kNG + 2 * t + 1] = st.l[1];
  }
  named_barrier_sync(1, 32 * kB8Warps);
  if (!KVQ_IN(slot >= 0 && slot < (DIRECT ? (int64_t)p.batch * p.hq : p.n_slots), p.flag)) return;
  for (int idx = tid; idx < p.g * (D / 4); idx += 32 * kB8Warps) {
    const int r = idx / (D / 4), c4 = idx % (D / 4);
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kB8Warps; ++w) mx = fmaxf(mx, sm.flush_m[w * kNG + r]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.0f;
    if (mx != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kB8Warps; ++w) {
        const float mw = sm.flush_m[w * kNG + r];
        const float f = mw == -INFINITY ? 0.0f : fast_exp2(mw - mx);
        const float4 x = *(reinterpret_cast<const float4*>(sm.flush_o + (w * kNG + r) * D) + c4);
        o.x = fmaf(f, x.x, o.x);
        o.y = fmaf(f, x.y, o.y);
        o.z = fmaf(f, x.z, o.z);
        o.w = fmaf(f, x.w, o.w);
        l = fmaf(f, sm.flush_l[w * kNG + r], l);
      }
    }
    if constexpr (DIRECT) {
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      store_out8(p, slot + r, D, c4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
      continue;
    }
    *(reinterpret_cast<float4*>(p.part_o + (slot * p.g + r) * D) + c4) = o;
    if (c4 == 0) *(reinterpret_cast<float2*>(p.part_ml) + slot * p.g + r) = make_float2(mx, l);
  }
}

// plan() for up to 32 sequences and a line that 32 bits count: one scan, 32-bit
// divisions; `per` is the ranges' length.  (plan() takes 2500 cycles here, this
// one 1500: 8 x 4096 positions, 32 query heads 18.8 -> 18.2 us; 4 x 1000 7.4 -> 6.8.)
template <int CHUNK>
__device__ __forceinline__ bool plan_short(const Decode8Params& p, uint32_t idx, uint32_t count, int64_t& v0,
                                           int64_t& v1, int64_t& per_out, Walker& wk) {
  if (p.batch > 32) return false;
  const int lane = threadIdx.x & 31;
  const uint32_t n = lane < p.batch ? (uint32_t)fp4_chunks<CHUNK>(walk_len(p, lane), 0) : 0u;
  // (32 sequences of < 2^25 / hkv chunks: no sum passes 2^30)
  if (__any_sync(0xFFFFFFFFu, n >= (1u << 25) / (uint32_t)p.hkv)) return false;
  const uint32_t x = n * (uint32_t)p.hkv;
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  const uint32_t total = __shfl_sync(0xFFFFFFFFu, incl, 31);
  const uint32_t per = (total + count - 1) / count;
  per_out = per;
  const uint32_t a = min(total, idx * per);
  v0 = a;
  v1 = min(total, a + per);
  wk.v = v0;
  if (v0 >= v1) return true;
  const int L = __ffs(__ballot_sync(0xFFFFFFFFu, incl > a)) - 1;
  const uint32_t nL = __shfl_sync(0xFFFFFFFFu, n, L), rem = a - __shfl_sync(0xFFFFFFFFu, incl - x, L);
  wk.b = L;
  wk.nch = (int)nL;
  wk.h = (int)(rem / nL);
  wk.c = (int)(rem - (uint32_t)wk.h * nL);
  return true;
}

// DIRECT: one CTA per unit, which walks all of its chunks and writes the result
// itself (caches of few chunks); else the equal ranges and partials described
// above.
template <int D, int GT, bool DIRECT, bool TEST>
__global__ void __launch_bounds__(kB8Threads, ctas8<D>()) decode_block8_kernel(const Decode8Params p) {
  using G = Geo8<D>;
  extern __shared__ uint8_t smem8_raw[];
  Smem8<D> sm = carve8<D>(smem8_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages8<D>(); ++s) {
      mbar_init(smem_addr(&sm.full[s]), 1);
      mbar_init(smem_addr(&sm.empty[s]), 32 * kB8Warps);
    }
    *sm.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  // Launched as a programmatic dependent of whatever precedes it on the
  // stream: every thread waits for that grid (the append of this step, the
  // previous step's merge still reading the workspace) before its first access
  // to global memory.
  grid_dependency_wait();

  int64_t v0, v1, per = 1;  // per: length of a range
  Walker wk;
  if constexpr (DIRECT) {
    wk.b = (int)(blockIdx.x / (unsigned)p.hkv);
    wk.h = (int)(blockIdx.x % (unsigned)p.hkv);
    const int32_t T = walk_len(p, wk.b);
    wk.c = 0;
    wk.v = v0 = 0;
    v1 = wk.nch = fp4_chunks<chunk8<D>()>(T, 0);
    if (v1 == 0) {  // no position: zero rows
      if (T < 0 && wk.h == 0 && threadIdx.x == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
      for (int i = threadIdx.x; i < p.g * (D / 4); i += kB8Threads)
        store_out8(p, (int64_t)wk.b * p.hq + (int64_t)wk.h * p.g + i / (D / 4), D, i % (D / 4),
                   make_float4(0.f, 0.f, 0.f, 0.f));
      return;
    }
  } else if (!plan_short<chunk8<D>()>(p, blockIdx.x, gridDim.x, v0, v1, per, wk)) {
    int64_t total;
    plan<chunk8<D>()>(p, blockIdx.x, gridDim.x, total, v0, v1, wk);
    per = (total + gridDim.x - 1) / gridDim.x;
  }
  if (v0 >= v1) return;
  if (warp == kB8Warps) {
    producer8<D, GT, TEST>(p, sm, wk, v1);
    return;
  }
  const uint32_t stages = smem_addr(sm.stages);
  State8<D> st;
  bool have = false, dead = false;
  int64_t slot = 0;
  uint32_t it = 0;
  for (; wk.v < v1; advance<chunk8<D>()>(p, wk), ++it) {
    if (!have || wk.c == 0) {
      uint2 rows[D / 16];
      load_rows8<D>(p, rows, wk.b, wk.h);
      if (!DIRECT && have) flush_unit8<D, DIRECT>(p, st, sm, slot);
      const int64_t u = (int64_t)wk.b * p.hkv + wk.h;
      slot = DIRECT ? u * p.g : u + blockIdx.x;  // (u * g: the unit's first output row)
      begin_unit8<D>(p, st, rows);
      have = true;
      if (!DIRECT && wk.c == 0 && threadIdx.x == 0) {
        const int64_t last_cta = (wk.v + wk.nch - 1) / per;
        if (KVQ_IN(u < (int64_t)p.batch * p.hkv && last_cta < gridDim.x, p.flag))
          p.unit_rec[u] = make_int2((int)slot, (int)(last_cta - blockIdx.x + 1));
      }
    }
    if (dead) continue;
    const uint32_t s = it % stages8<D>();
    bool ok = !*reinterpret_cast<volatile int*>(sm.abort) && work_wait8<TEST>(p, smem_addr(&sm.full[s]), (it / stages8<D>()) & 1);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) {
      dead = true;
      if (lane == 0) {
        set_flag(p.flag, KVQ_FLAG_TIMEOUT);
        *reinterpret_cast<volatile int*>(sm.abort) = 1;
      }
      continue;
    }
    const int ntok = sm.ntok[s];
    const uint32_t good = sm.good[s], bar = smem_addr(&sm.empty[s]), stage = stages + s * G::kStageBytes;
    const int s0 = warp * G::kSlices;
    constexpr uint32_t kAll = (1u << G::kSlices) - 1u;
    if (ntok >= 16 * (s0 + G::kSlices) && ((good >> s0) & kAll) == kAll) {
      if constexpr (G::kSlices > 1) consume8<D, GT, false, false>(st, stage, s0, 16, bar);
      consume8<D, GT, false, true>(st, stage, s0 + G::kSlices - 1, 16, bar);
    } else {
#pragma unroll 1
      for (int i = s0; i < s0 + G::kSlices; ++i)
        if (ntok > 16 * i && ((good >> i) & 1u)) consume8<D, GT, true, false>(st, stage, i, ntok - 16 * i, bar);
      mbar_arrive(bar);
    }
  }
  if (have) flush_unit8<D, DIRECT>(p, st, sm, slot);
}

// ------------------------------------------------------------------ host side
template <int D, int GT, bool DIRECT, bool TEST>
kvq_status launch_decode8(const Decode8Params& dp, cudaStream_t s, int ctas) {
  static DeviceOnce attr_set;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
  if (attr_set.pending(dev)) {
    if (cudaFuncSetAttribute(decode_block8_kernel<D, GT, DIRECT, TEST>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Geo8<D>::kSmemBytes) != cudaSuccess)
      return KVQ_ERR_CUDA;
    attr_set.mark(dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kB8Threads);
  cfg.dynamicSmemBytes = (size_t)Geo8<D>::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_block8_kernel<D, GT, DIRECT, TEST>, dp) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

template <int D, bool DIRECT>
kvq_status launch_decode8_d(const Decode8Params& dp, cudaStream_t s, int ctas) {
  switch (dp.c.page_size) {
    case 16: return launch_decode8<D, 16, DIRECT, false>(dp, s, ctas);
    case 32: return launch_decode8<D, 32, DIRECT, false>(dp, s, ctas);
    default: break;
  }
  return dp.wait_ns == 0 ? launch_decode8<D, 64, DIRECT, false>(dp, s, ctas) : launch_decode8<D, 64, DIRECT, true>(dp, s, ctas);
}

// One CTA per unit, without partials and their merge, when the cache's capacity
// (which the host knows; the lengths it does not) holds few chunks per unit, or
// not many and units for every SM.  Both ways, us a call, 8 kv heads of 128:
//   batch 8:   512 positions 6.8 direct, 7.4 split;  1024: 10.8, 8.7;  2048: 19.8, 12.3
//   batch 32:  512           8.7,        12.9;       1024: 14.8, 19.2; 2048: 24.5, 29.0
constexpr int kDirectChunks = 8, kDirectChunksFull = 32;

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_fp8_block_decode_attn(const kvq_cache* cache, int32_t batch, int32_t num_q_heads,
                                                const int32_t* d_seq_lens, const void* q, float softmax_scale,
                                                void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                                int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 1) return KVQ_ERR_INVALID_ARGUMENT;
  kvq_status st = check_block8_cache(cache, batch);
  if (st != KVQ_OK) return st;
  const int hkv = cache->num_kv_heads, D = cache->head_dim;
  if (num_q_heads < hkv || num_q_heads % hkv != 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (!(softmax_scale > 0.0f) || !(softmax_scale < 3.0e38f)) return KVQ_ERR_INVALID_ARGUMENT;
  if (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16) return KVQ_ERR_INVALID_ARGUMENT;
  if (d_seq_lens == nullptr || q == nullptr || out == nullptr || workspace == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(workspace, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  const int g = num_q_heads / hkv;
  if (g > kNG) return KVQ_ERR_UNSUPPORTED;
  const int64_t units = (int64_t)batch * hkv;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  // the workspace is laid out for three CTAs per SM, as kvq_decode_attn's
  const int64_t n_slots = units + 3 * (int64_t)sms;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t ml_off = up((size_t)units * sizeof(int2));
  const size_t o_off = ml_off + up((size_t)n_slots * g * 2 * sizeof(float));
  if (workspace_bytes < o_off + up((size_t)n_slots * g * D * sizeof(float))) return KVQ_ERR_WORKSPACE;
  // a persistent grid; for a cache whose capacity holds little, no more CTAs
  // than have two chunks each (4 x 1000 positions, 8 kv heads: 8.0 -> 7.5 us,
  // with fewer partials to merge)
  const int64_t cap = (int64_t)cache->max_pages_per_seq * cache->page_size;
  const int chunk = D == 128 ? chunk8<128>() : chunk8<64>();
  const int64_t unit_chunks = (cap + chunk - 1) / chunk;
  const int64_t pairs = (units * unit_chunks + 1) / 2;
  const int64_t full = (int64_t)sms * (D == 128 ? ctas8<128>() : ctas8<64>());
  const int ctas = (int)(pairs < full ? pairs : full);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  Decode8Params dp = {};
  dp.lens = d_seq_lens;
  dp.c = *cache;
  dp.q = static_cast<const uint16_t*>(q);
  dp.unit_rec = reinterpret_cast<int2*>(ws);
  dp.part_ml = reinterpret_cast<float*>(ws + ml_off);
  dp.part_o = reinterpret_cast<float*>(ws + o_off);
  dp.flag = d_err_flag;
  dp.batch = batch;
  dp.hkv = hkv;
  dp.g = g;
  dp.hq = num_q_heads;
  dp.qk_log2 = softmax_scale * kLog2e;
  dp.n_slots = n_slots;
  dp.wait_ns = test_wait_limit_ns();
  if (units <= INT32_MAX &&
      (unit_chunks <= kDirectChunks || (unit_chunks <= kDirectChunksFull && units >= (int64_t)sms))) {
    dp.out = out;
    dp.out_bf16 = out_dtype == KVQ_DTYPE_BF16;
    return D == 128 ? launch_decode8_d<128, true>(dp, s, (int)units) : launch_decode8_d<64, true>(dp, s, (int)units);
  }
  st = D == 128 ? launch_decode8_d<128, false>(dp, s, ctas) : launch_decode8_d<64, false>(dp, s, ctas);
  if (st != KVQ_OK) return st;

  MergeParams mp = {};
  mp.lens = d_seq_lens;
  mp.q = dp.q;
  mp.part_o = dp.part_o;
  mp.part_ml = dp.part_ml;
  mp.unit_rec = dp.unit_rec;
  mp.out = out_dtype == KVQ_DTYPE_F32 ? static_cast<float*>(out) : nullptr;
  mp.out_bf16 = out_dtype == KVQ_DTYPE_BF16 ? static_cast<uint16_t*>(out) : nullptr;
  mp.flag = d_err_flag;
  mp.hkv = hkv;
  mp.g = g;
  mp.hq = num_q_heads;
  mp.head_dim = D;
  mp.qk_log2 = dp.qk_log2;
  mp.n_slots = n_slots;
  mp.batch = batch;
  return launch_merge(mp, units, s);
}
