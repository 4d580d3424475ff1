// kvq_expanded_attn.cu -- causal attention of a chunk over dense keys and values
// whose key's position part is shared by all heads, on the 5th-generation tensor
// cores (tcgen05, accumulators in TMEM), and its C entry point.
//
// Mathematics.  Query token i of n sits at position T - n + i and attends 0 .. T - n + i,
//   S = q[:d] . k + q[d:] . k_rope,  P = 2^(f S - m),  f = softmax_scale log2 e,
//   out = sum P v / sum P.
// q, k and v enter the products as they are (bf16); P is rounded to bf16, which has
// fp32's range; sums, maxima and accumulators are fp32.  The reference m of a row is raised
// only when a score passes the one it was set by by more than kSlackE, and lies so far over
// that one that no sum of the unit's P reaches past 1: 8 for the slack and log2 of the
// positions.  So sum P v stays within fp32's range for every finite v (the largest bf16 values
// leave no factor at all), at the other end's cost: products under 2^-126 are lost.
// Where f times that score is over 2^27, m's rounding would stand in P (2^7 in its exponent at
// 2^31), but neighbouring fp32 scores lie 2^8 in P and more apart: the row takes a power of two
// for f, for which f S and m, then without the room, are exact.
//
// What bounds it: the tensor pipe, 2 (2 d + 64) flop per attended pair and head; a
// unit's tiles come from L2, 51 KB per 80 positions at d = 128.
// Work: a CTA takes 256 query tokens of a head as two 128-row tiles that share each
// tile of 80 positions: with 80, tensor memory holds both tiles' scores, weights and
// sums side by side, so that the next scores are computed beside the softmax of these
// (with 96 and the weights over the scores: S, softmax and P V one after the other, 3200
// cycles a tile; 302 us where this takes 277, 2 x 4096 tokens, 32 heads of 128).  The longest first, 16 heads at a time so that their keys and
// values stay in L2.
// Twelve warps: softmax (2 x 4, thread = row), loader (TMA, 128-byte swizzle), MMA
// issue (one per query tile, so that one's softmax runs beside the other's products),
// values, joined by mbarriers (every wait bounded):
//   S_X(j) = q_X K(j)^T    both from shared memory; the key's position part is one
//                          more 64-channel slab behind the head's own
//   O_X += P_X(j) V(j)     P from TMEM, V as MN-major operand
//                          in the order S(j + 1), O(j)
//   values                 in tiles that some row attends in part (five of a unit at most)
//                          Inf and NaN leave V, since a weight of 0 would carry them to
//                          rows that do not see them, and are noted by channel: the rows
//                          from the first one's position on are NaN there
#include "../../include/kvq_latent.h"
#include "kvq_common.cuh"
#include "kvq_host.cuh"
#include "kvq_roles.cuh"
#include "kvq_tc.cuh"

#include <cuda_bf16.h>

namespace kvq {
namespace {

constexpr int kET = 80;       // positions per tile
constexpr int kERows = 128;   // rows of a query tile
constexpr int kERope = 64;
constexpr int kESoftmax = 8, kELoad = kESoftmax, kEMma = kELoad + 1, kEValues = kEMma + 2, kEThreads = 32 * (kEValues + 1);
constexpr int kQSlab = kERows * 128, kTSlab = kET * 128;  // 64 channels of a query tile, of a tile
constexpr int kHeadsAtOnce = 16;
constexpr float kSlackE = 8.0f;

enum : int {
  kEQ = 0,              // queries landed
  kEKFull = 1,          // [ring]
  kEKEmpty = kEKFull + 4,
  kEVFull = kEKEmpty + 4,
  kEVEmpty = kEVFull + 4,
  kEVIn = kEVEmpty + 4,     // [ring] a partly attended tile's values landed (kEVFull: looked at, too)
  kESFull = kEVIn + 4,      // [2] S_X in TMEM
  kESFree = kESFull + 2,    // [2] S_X taken by the softmax
  kEPFull = kESFree + 2,    // [2] P_X in TMEM, O_X rescaled
  kEPvDone = kEPFull + 2,   // [2] O_X += done
  kEDrain = kEPvDone + 2,   // [2] an MMA warp's last commit
  kEBars = kEDrain + 2
};

struct ExpandedParams {
  const int32_t* lens;
  const int32_t* chunk_lens;
  void* out;
  int32_t* flag;
  int32_t batch, heads, chunk, max_len, out_bf16, nqb;
  float scale_log2;
  uint64_t wait_ns;  // a test's limit of the waits, or 0
};

template <int D>
struct EGeo {
  static constexpr int kKSlabs = (D + kERope) / 64, kVSlabs = D / 64;
  static constexpr int kRing = D == 128 ? 2 : 4;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kKSlabs * kQSlab;
  static constexpr int kV = kK + kRing * kKSlabs * kTSlab;
  static constexpr int kBar = kV + kRing * kVSlabs * kTSlab;
  static constexpr int kNan = kBar + 8 * kEBars;  // [D] the first position whose value is Inf or NaN
  static constexpr int kMisc = kNan + 4 * D;
  static constexpr int kBytes = kMisc + 16 + 1024;  // 1024: the swizzle's alignment
  static constexpr int kSCol = 2 * D, kPCol = kSCol + 2 * kET;  // O_X at [X D, +D)
  static_assert(kBytes <= 227 * 1024 && kBytes > 116 * 1024 && kPCol + kET <= 512, "layout");
};

// Descriptors of operands with the 128-byte swizzle (8 rows of 128 bytes an atom).
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return smem_desc(saddr, lbo, sbo) | (uint64_t)2 << 61;
}
// kind::f16, bf16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// 16 columns of this warp's TMEM lanes and their maximum, without the wait.
__device__ __forceinline__ void tmem_ld_max16(uint32_t taddr, uint32_t* v, uint32_t& m) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, "
      "[%17];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(m)
      : "r"(taddr)
      : "memory");
}
// 8 columns of this warp's TMEM lanes, without the wait.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// keeps the uses of v and m behind the wait
__device__ __forceinline__ void behind(uint32_t* v, uint32_t& m) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(m)
               :
               : "memory");
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kEThreads, 1)
    expanded_attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mr, const __grid_constant__ CUtensorMap mv,
                         const ExpandedParams p) {
  using G = EGeo<D>;
  extern __shared__ uint8_t exp_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(exp_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(base), bars = sb + G::kBar;
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + G::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 1);
  const BoundedWaits wait{abort, p.wait_ns};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // 16 heads at a time, within them the last tokens (the longest) first
  const int bhs = p.batch * p.heads, part = blockIdx.x / (kHeadsAtOnce * p.nqb);
  const int in_part = min(kHeadsAtOnce, bhs - part * kHeadsAtOnce), at = blockIdx.x - part * kHeadsAtOnce * p.nqb;
  const int bh = part * kHeadsAtOnce + at % in_part, qb = p.nqb - 1 - at / in_part;
  const int h = bh % p.heads, b = bh / p.heads;
  const int32_t T = __ldg(p.lens + b), n = p.chunk_lens ? __ldg(p.chunk_lens + b) : p.chunk;
  if (n < 0 || n > p.chunk || T > p.max_len || T < n) {
    if (tid == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
    if (n < 0 || n > p.chunk || T > p.max_len) return;
  }
  const int i0 = qb * 2 * kERows;
  if (i0 >= n) return;  // padding only
  const int rows = min(2 * kERows, n - i0);
  const int64_t row0 = ((int64_t)b * p.chunk + i0) * p.heads + h;
  if (T < n) {  // the chunk's own tokens must be among the keys
    for (int i = tid; i < rows * (D / 4); i += kEThreads) {
      const int64_t o = (row0 + (int64_t)(i / (D / 4)) * p.heads) * D + i % (D / 4) * 4;
      if (p.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) = make_uint2(0u, 0u);
      else
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const int first = T - n + i0;                  // position of the unit's token 0
  const int nx = rows > kERows ? 2 : 1;          // query tiles with rows
  // tiles that query tile X attends
  const auto tiles_of = [&](int x) { return (first + min(rows, kERows * (x + 1)) + kET - 1) / kET; };
  const int nt = tiles_of(nx - 1);
  const int part0 = (first + 1) / kET;           // the first tile that not all rows attend

  if (tid == 0) {
    mbar_init(bars + 8 * kEQ, 1);
    for (int i = 0; i < G::kRing; ++i) {
      mbar_init(bars + 8 * (kEKFull + i), 1);
      mbar_init(bars + 8 * (kEKEmpty + i), nx);
      mbar_init(bars + 8 * (kEVFull + i), 1);
      mbar_init(bars + 8 * (kEVEmpty + i), nx);
      mbar_init(bars + 8 * (kEVIn + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (kESFull + i), 1);
      mbar_init(bars + 8 * (kESFree + i), 4);
      mbar_init(bars + 8 * (kEPFull + i), 4);
      mbar_init(bars + 8 * (kEPvDone + i), 1);
      mbar_init(bars + 8 * (kEDrain + i), 1);
    }
    *abort = 0;
    misc[2] = 0u;
    fence_barrier_init();
  }
  int* nan_first = reinterpret_cast<int*>(base + G::kNan);
  if (tid < D) nan_first[tid] = INT32_MAX;
  if (warp == 0) tmem_alloc(smem_addr(misc), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);

  // where tile j's values land, and the phase of that
  const auto values_in = [&](int j) { return bars + 8 * ((j < part0 ? kEVFull : kEVIn) + j % G::kRing); };
  const auto values_phase = [&](int j) { return (uint32_t)((j < part0 ? j : j - part0) / G::kRing) & 1u; };

  if (warp < kESoftmax) {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2, r = tid & 127, i = kERows * x + r;
    const uint32_t tw = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = tw + G::kSCol + x * kET, p_col = tw + G::kPCol + x * (kET / 2), o_col = tw + x * D;
    const int ntx = x < nx ? tiles_of(x) : 0;
    const int last = first + i, all = first + kERows * x;  // last position of the row, of every row
    const float room = (float)(32 - __clz(first + rows - 1)) + kSlackE;  // (log2 of the positions, rounded up)
    // the score that set the row's m, the one that a larger one has to pass to raise it, f and m
    float ref = -INFINITY, past = -INFINITY, f = p.scale_log2, m = room;
    uint64_t l2 = 0ull;
    bool ok = true;
    for (int j = 0; j < ntx && ok; ++j) {
      if (!(ok = wait(bars + 8 * (kESFull + x), j & 1u))) break;
      tc_fence_after();
      uint32_t v[kET], mx[kET / 16];
#pragma unroll
      for (int k = 0; k < kET / 16; ++k) tmem_ld_max16(s_col + 16 * k, v + 16 * k, mx[k]);
      asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
      for (int k = 0; k < kET / 16; ++k) behind(v + 16 * k, mx[k]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (kESFree + x));
      float top = -INFINITY;
      if ((j + 1) * kET > all + 1) {  // some row sees the tile in part
        const int lim = last - j * kET;
#pragma unroll
        for (int c = 0; c < kET; ++c) {
          if (c > lim) v[c] = 0xFF800000u;
          top = fmaxf(top, __uint_as_float(v[c]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < kET / 16; ++k) top = fmaxf(top, __uint_as_float(mx[k]));
      }
      // the sums of the tile before: done with O and P
      if (j > 0 && !(ok = wait(bars + 8 * (kEPvDone + x), (j - 1) & 1u))) break;
      tc_fence_after();
      const bool up = top > past;
      if (__any_sync(0xFFFFFFFFu, up)) {
        float a = 1.0f;
        if (up) {
          const float y = fabsf(top * p.scale_log2), old = f, m_old = m;
          const bool far = y > 134217728.0f;
          f = far ? __uint_as_float((__float_as_uint(p.scale_log2) + 0x400000u) & 0x7F800000u) : p.scale_log2;
          m = fmaf(top, f, far ? 0.0f : y > 16384.0f ? room + 4.0f : room);  // (4: half its steps under 2^27)
          a = ref == -INFINITY ? 0.0f : fast_exp2(fmaf(ref, f, -m) - fmaf(ref, old, -m_old));
          ref = top;
          past = __fadd_rd(ref, kSlackE / p.scale_log2);
        }
        l2 = mul2(l2, pack2(a, a));
        if (j > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_col + c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            tmem_st32_async(o_col + c, o);
          }
        }
      }
      const uint64_t c2 = pack2(f, f), r2 = pack2(-m, -m);
#pragma unroll
      for (int k = 0; k < kET / 16; ++k) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = 16 * k + 2 * e;
          const float2 y = unpack2(fma2(pack2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), c2, r2));
          const float a = fast_exp2(y.x), bb = fast_exp2(y.y);
          l2 = add2(l2, pack2(a, bb));
          w[e] = bf16x2(a, bb);
        }
        tmem_st8(p_col + 8 * k, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (kEPFull + x));
    }
    if (ok && ntx > 0 && (ok = wait(bars + 8 * (kEPvDone + x), (ntx - 1) & 1u))) {
      tc_fence_after();
      const float2 ll = unpack2(l2);
      const float l = ll.x + ll.y, f = 1.0f / l;  // (l is 0 where every score is -Inf: 0 * Inf, a row of NaN)
      const int64_t o = (row0 + (int64_t)i * p.heads) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t w[32];
        tmem_ld32(o_col + c, w);
        if (i < rows) {
#pragma unroll
          for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
          if (*reinterpret_cast<volatile uint32_t*>(misc + 2)) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (nan_first[c + k] <= last) w[k] = 0x7FFFFFFFu;
          }
          if (p.out_bf16) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + o + c + k) =
                  make_uint4(bf16x2(__uint_as_float(w[k]), __uint_as_float(w[k + 1])),
                             bf16x2(__uint_as_float(w[k + 2]), __uint_as_float(w[k + 3])),
                             bf16x2(__uint_as_float(w[k + 4]), __uint_as_float(w[k + 5])),
                             bf16x2(__uint_as_float(w[k + 6]), __uint_as_float(w[k + 7])));
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + o + c + k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
          }
        }
      }
    }
  } else if (warp == kELoad) {
    // ------------------------------------------------------------ loader
    if (lane == 0) {
      mbar_arrive_expect_tx(bars + 8 * kEQ, nx * G::kKSlabs * kQSlab);
      for (int x = 0; x < nx; ++x)
        for (int s = 0; s < G::kKSlabs; ++s)
          tma_4d(sb + G::kQ + (x * G::kKSlabs + s) * kQSlab, &mq, 64 * s, h, i0 + kERows * x, b, bars + 8 * kEQ);
    }
    __syncwarp();
    int kj = 0, vj = 0;  // tiles so far
    for (int j = 0; j < nt; ++j) {
      const int s = j % G::kRing;
      if (j >= G::kRing && !wait(bars + 8 * (kEKEmpty + s), (uint32_t)(j / G::kRing - 1) & 1u)) break;
      if (lane == 0) {
        const uint32_t bar = bars + 8 * (kEKFull + s), dst = sb + G::kK + s * G::kKSlabs * kTSlab;
        mbar_arrive_expect_tx(bar, G::kKSlabs * kTSlab);
        for (int c = 0; c < D / 64; ++c) tma_4d(dst + c * kTSlab, &mk, 64 * c, h, j * kET, b, bar);
        tma_load_3d(dst + D / 64 * kTSlab, &mr, 0, j * kET, b, bar);
      }
      __syncwarp();
      kj = j + 1;
      if (j >= G::kRing && !wait(bars + 8 * (kEVEmpty + s), (uint32_t)(j / G::kRing - 1) & 1u)) break;
      if (lane == 0) {
        const uint32_t bar = values_in(j), dst = sb + G::kV + s * G::kVSlabs * kTSlab;
        mbar_arrive_expect_tx(bar, G::kVSlabs * kTSlab);
        for (int c = 0; c < G::kVSlabs; ++c) tma_4d(dst + c * kTSlab, &mv, 64 * c, h, j * kET, b, bar);
      }
      __syncwarp();
      vj = j + 1;
    }
    // no copy outlives the CTA
    const auto landed = [&](uint32_t bar, uint32_t parity) {
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait_hint(bar, parity, 20000u) && global_ns() - t0 < 20000000ull) {
      }
    };
    landed(bars + 8 * kEQ, 0u);
    for (int j = max(0, kj - G::kRing); j < kj; ++j) landed(bars + 8 * (kEKFull + j % G::kRing), (uint32_t)(j / G::kRing) & 1u);
    for (int j = max(0, vj - G::kRing); j < vj; ++j) landed(values_in(j), values_phase(j));
  } else if (warp - kEMma < nx) {
    // ------------------------------------------------------------ MMA issue
    const int x = warp - kEMma, ntx = tiles_of(x);
    const uint64_t dq = swizzled_desc(sb + G::kQ + x * G::kKSlabs * kQSlab, 16, 1024);
    const uint64_t dk = swizzled_desc(sb + G::kK, 16, 1024);        // positions as rows: K-major
    const uint64_t dv = swizzled_desc(sb + G::kV, kTSlab, 1024);    // channels as rows: MN-major
    const uint32_t s_col = tmem + G::kSCol + x * kET, p_col = tmem + G::kPCol + x * (kET / 2), o_col = tmem + x * D;
    const auto scores = [&](int j) {
      const int s = j % G::kRing;
      if (elect_one_of_warp()) {
        const uint64_t k0 = dk + (uint64_t)(s * (G::kKSlabs * kTSlab >> 4));
#pragma unroll
        for (int c = 0; c < (D + kERope) / 16; ++c)
          tc_mma_f16(s_col, dq + (uint64_t)(((c >> 2) * kQSlab + (c & 3) * 32) >> 4),
                     k0 + (uint64_t)(((c >> 2) * kTSlab + (c & 3) * 32) >> 4), idesc_bf16(kET, false), c > 0);
        tc_commit(bars + 8 * (kESFull + x));
        tc_commit(bars + 8 * (kEKEmpty + s));
      }
      __syncwarp();
    };
    bool ok = wait(bars + 8 * kEQ, 0u) && wait(bars + 8 * kEKFull, 0u);
    tc_fence_after();
    if (ok) scores(0);
    for (int j = 0; j < nt && ok; ++j) {
      const int s = j % G::kRing, sn = (j + 1) % G::kRing;
      const uint32_t ph = (uint32_t)(j / G::kRing) & 1u, phn = (uint32_t)((j + 1) / G::kRing) & 1u;
      if (j + 1 < nt) {
        if (!(ok = wait(bars + 8 * (kEKFull + sn), phn))) break;
        if (j + 1 < ntx) {
          if (!(ok = wait(bars + 8 * (kESFree + x), j & 1u))) break;
          tc_fence_after();
          scores(j + 1);
        } else if (lane == 0) {  // a tile that only the other query tile attends
          mbar_arrive(bars + 8 * (kEKEmpty + sn));
        }
      }
      if (!(ok = wait(bars + 8 * (kEVFull + s), ph))) break;
      if (j < ntx) {
        if (!(ok = wait(bars + 8 * (kEPFull + x), j & 1u))) break;
        tc_fence_after();
        if (elect_one_of_warp()) {
          const uint64_t v0 = dv + (uint64_t)(s * (G::kVSlabs * kTSlab >> 4));
#pragma unroll
          for (int c = 0; c < kET / 16; ++c)
            tc_mma_f16_ta(o_col, p_col + 8 * c, v0 + (uint64_t)(c * 2048 >> 4), idesc_bf16(D, true), j > 0 || c > 0);
          tc_commit(bars + 8 * (kEPvDone + x));
          tc_commit(bars + 8 * (kEVEmpty + s));
        }
        __syncwarp();
      } else if (lane == 0) {
        mbar_arrive(bars + 8 * (kEVEmpty + s));
      }
    }
    // no product outlives the CTA (a commit covers its own thread's, so the lane that issued them makes it)
    __syncwarp();
    if (elect_one_of_warp()) tc_commit(bars + 8 * (kEDrain + x));
    __syncwarp();
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait_hint(bars + 8 * (kEDrain + x), 0u, 20000u) && global_ns() - t0 < 20000000ull) {
    }
  } else if (warp == kEValues) {
    // ------------------------------------------------------------ values
    for (int j = part0; j < nt; ++j) {
      const int s = j % G::kRing;
      if (!wait(values_in(j), values_phase(j))) break;
      const uint32_t v0 = sb + G::kV + s * G::kVSlabs * kTSlab;
      const int there = T - j * kET;  // positions of the tile that the sequence has
      uint32_t top = 0u;              // the largest magnitudes' bits, Inf and NaN above the rest
#pragma unroll 8
      for (int k = 0; k < G::kVSlabs * kET / 4; ++k) {
        const uint4 v = lds128(v0 + 512 * k + 16 * lane);
        top = max_u16x2(max_u16x2(top, v.x & 0x7FFF7FFFu), max_u16x2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu));
        top = max_u16x2(top, v.w & 0x7FFF7FFFu);
      }
      const bool look = (top & 0xFFFFu) >= 0x7F80u || top >= 0x7F800000u || there < kET;
      bool found = false;
      if (__any_sync(0xFFFFFFFFu, look))
#pragma unroll 1
      for (int k = lane; k < G::kVSlabs * kET * 8; k += 32) {  // 16-byte units: slab, position, eight channels
        const int pos = k / 8 % kET, slab = k / (8 * kET);
        const uint32_t at = v0 + slab * kTSlab + k % (8 * kET) * 16;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        uint32_t bad = pos < there ? 0u : 1u;
        if (pos < there) {
          v = lds128(at);
          uint32_t* w = &v.x;
          uint32_t hit = 0u;  // bit c: channel c of the eight
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if ((w[c] & 0x7F80u) == 0x7F80u) hit |= 1u << 2 * c, w[c] &= 0xFFFF0000u;
            if ((w[c] & 0x7F800000u) == 0x7F800000u) hit |= 2u << 2 * c, w[c] &= 0xFFFFu;
          }
          bad = hit;
          const int ch = 64 * slab + (k % 8 ^ (pos & 7)) * 8;  // (the swizzle's place of the unit)
          for (; hit; hit &= hit - 1u) {
            atomicMin(nan_first + ch + __ffs(hit) - 1, j * kET + pos);
            found = true;
          }
        }
        if (bad) sts128(at, v);
      }
      if (found) *reinterpret_cast<volatile uint32_t*>(misc + 2) = 1u;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (kEVFull + s));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort) set_flag(p.flag, KVQ_FLAG_TIMEOUT);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool rows_ok(int64_t token, int64_t head, int64_t heads, int64_t width) {
  if (token % 8 != 0 || head % 8 != 0 || head < 0 || token < 0) return false;
  return (heads <= 1 || head >= width) && token >= (heads - 1) * head + width;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// bf16 rows of `width` values, [batch][tokens][heads] (heads 0: no such dimension),
// copied by boxes of 64 values x `box` tokens of one head.
bool encode(CUtensorMap* map, const void* ptr, int64_t width, int64_t heads, int64_t tokens, int64_t batch, int64_t head_stride,
            int64_t token_stride, int box) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const int rank = heads ? 4 : 3;
  cuuint64_t dims[4], strides[3];
  cuuint32_t boxes[4], steps[4] = {1, 1, 1, 1};
  int d = 0;
  dims[d] = (cuuint64_t)width, boxes[d++] = 64;
  if (heads) strides[d - 1] = (cuuint64_t)head_stride * 2, dims[d] = (cuuint64_t)heads, boxes[d++] = 1;
  strides[d - 1] = (cuuint64_t)token_stride * 2, dims[d] = (cuuint64_t)tokens, boxes[d++] = (cuuint32_t)box;
  strides[d - 1] = (cuuint64_t)token_stride * 2 * (cuuint64_t)tokens, dims[d] = (cuuint64_t)batch, boxes[d++] = 1;
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, boxes, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
kvq_status launch_expanded(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mr, const CUtensorMap& mv,
                           const ExpandedParams& p, cudaStream_t s) {
  static DeviceOnce attr_set;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
  if (attr_set.pending(dev)) {
    if (cudaFuncSetAttribute(expanded_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, EGeo<D>::kBytes) != cudaSuccess)
      return KVQ_ERR_CUDA;
    attr_set.mark(dev);
  }
  expanded_attn_kernel<D><<<(unsigned)((int64_t)p.batch * p.heads * p.nqb), kEThreads, EGeo<D>::kBytes, s>>>(mq, mk, mr, mv, p);
  return launch_status();
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
      rope_dim != kERope || !(softmax_scale > 0.0f) || !(softmax_scale < 2.0e38f) ||
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
  ExpandedParams p = {};
  p.nqb = (int32_t)(((int64_t)chunk + 2 * kERows - 1) / (2 * kERows));
  if ((double)batch * chunk * num_heads > (double)(1 << 30) || (double)batch * num_heads * p.nqb > (double)(1 << 30) ||
      max_len > (1 << 30))
    return KVQ_ERR_UNSUPPORTED;
  p.lens = d_seq_lens, p.chunk_lens = d_chunk_lens;
  p.out = out, p.flag = d_err_flag;
  p.batch = batch, p.heads = num_heads, p.chunk = chunk, p.max_len = max_len;
  p.out_bf16 = out_dtype == KVQ_DTYPE_BF16;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.wait_ns = test_wait_limit_ns();
  const int64_t w = head_dim + rope_dim;
  const int64_t tokens = max_len > 0 ? max_len : 1;  // (without keys nothing is copied: any map will do)
  const int64_t kh = num_heads > 1 ? k_head_stride : head_dim, vh = num_heads > 1 ? v_head_stride : head_dim;
  CUtensorMap mq, mk, mr, mv;
  if (!encode(&mq, q, w, num_heads, chunk, batch, w, w * num_heads, kERows) ||
      !encode(&mk, max_len > 0 ? k : q, head_dim, num_heads, tokens, batch, kh, k_token_stride, kET) ||
      !encode(&mr, max_len > 0 ? k_rope : q, rope_dim, 0, tokens, batch, 0, k_rope_stride, kET) ||
      !encode(&mv, max_len > 0 ? v : q, head_dim, num_heads, tokens, batch, vh, v_token_stride, kET))
    return KVQ_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch_expanded<128>(mq, mk, mr, mv, p, s) : launch_expanded<64>(mq, mk, mr, mv, p, s);
}
