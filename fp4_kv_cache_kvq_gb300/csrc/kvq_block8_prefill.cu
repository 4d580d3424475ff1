// kvq_block8_prefill.cu -- chunked-prefill attention over the 8-bit block
// cache on the 5th-generation tensor cores (tcgen05, accumulators in TMEM),
// and its C entry points.
//
// Mathematics.  Query token i of n sits at position T - n + i and attends
// 0 .. T - n + i.  With one K and one V scale per 16 positions,
//   S = q . code_K,  y = S (softmax_scale log2 e sK),  P = 2^(y + log2 sV - m'),
//   O = sum P code_V,  l = sum P / sV,  out = O / l.
// S takes the cached K codes as they are: q, scaled per row by a power of two
// to [2^7, 2^8), is the sum of two E4M3 values hi = RNE(q) and lo = q - hi
// (a bf16 value has 8 significant bits and an E4M3 value 4; lo, whose smallest step
// is 2^-9, is exact down to 2^-9 of the row's largest element and off by at most
// 2^-17 of it under that), so S = hi . K + lo . K are two fp8 products, which together cost one
// f16 product and need no expansion of K.  The V scale of a block goes into P's
// exponent, beside the softmax's own, so V^ is the codes themselves (exact in
// f16; a scale that is no power of two leaves its significand, [1, 2), to V^,
// rounded to f16 there).  P is rounded to f16: 2^-11 relative, or 2^-25 of 2^m',
// where m' is at most the largest y + log2 sV that the row has attended, rounded up.  So what
// a row loses is measured by what it attends itself, and no value behind its last
// position, however large, reaches it.  l takes P's fp32 value back to 2^(y - m),
// m a second reference, with one factor per block: weights on blocks of tiny values
// count in l although their P rounds to 0 (the exponent that V adds is held at -60
// and up for that, far under what f16 sees).  Both references are whole numbers, so
// every sum of exponents is exact.  Accumulation, maxima and sums are fp32.
// A block that a row sees in part can owe its scale to a token behind the row.  In a
// tile that some row sees in part, with a scale 2^kScaleSpread over the smallest so far,
// each token's own largest code therefore goes into P's exponent instead of its block's
// scale, and out of V^ (exactly, too).  NaN values of such a tile are taken out of V^
// (a product would carry them to the rows that do not see them) and noted by channel;
// the rows from the first one on are NaN there.
//
// What bounds it: the tensor pipe, 4 Hq d flop per attended pair.  Work split:
// a CTA takes 256 query rows (G heads x 256/G tokens) of one kv head as two
// 128-row tiles that share each 128-position cache tile; when few rows would
// leave SMs idle, the positions are split over several CTAs too and a second
// launch joins their partials.
// Sixteen warps: softmax (2 x 4, thread = row), V expansion (4), loader (1), MMA
// issue (one per query tile), scales (1), joined by mbarriers (every wait bounded):
//   loader    bulk copies of K codes, V codes and scales into rings of 3 tiles;
//             the pool's K layout is the tensor core's operand layout
//   MMA       S_X(j) = Qhi_X K(j)^T + Qlo_X K(j)^T   kind::f8f6f4
//             O_X += P_X(j) V^(j)                    kind::f16, P_X from TMEM
//             the two tiles in turn: O_A(j), S_A(j+1), O_B(j), S_B(j+1)
// Measured (1024 tokens over 16384 positions, 4 sequences, 64 query and 8 kv heads
// of 128, page 64; calls in a row, L2 flushed): 1485 us, 1.43 PFLOP/s, 0.75 of the bf16
// GEMM rate; 1560 us (0.71) among other kernels' calls.  head_dim 64: 1243.
// From 2.09 ms: a row's scores in registers with the maxima that the TMEM load takes
// 1.99; the issuing warp uniform 1.75; one issuing warp per query tile, in turns 1.67;
// the running maximum raised only past 2^15 1.52; queries read by four lanes a row and
// results stored through shared memory (a thread per row touches 32 lines an access),
// and no CTA-wide wait before the first product 1.46; a kernel of its own for pairs 1.41.
// What precision costs of that: V's scales in P's exponent instead of a factor relative
// to the largest of the CTA's positions 1407 -> 1450 us (head_dim 64: 1200 -> 1224), with
// what follows from the scales alone computed ahead of the scores, by one warp for all
// rows where it does not depend on the row (1493 behind the scores, 1466 by every row);
// the form with exponents for single tokens 1468 (1247), beside code that these cases do
// not enter (1505 with every partly attended tile looked at); the look for NaN values
// 1478 (1249).
// Before these, a tile of both query tiles took 2980 cycles, 2048 of them products: each
// query tile's chain was P V^ 890, S 890 (512 and a wait each), softmax 1090, and the
// other tile's filled the gaps.
// Slower: two threads per row 1.72; S of the next tile started before O of this
// one's turn ends 1.58; P stored in halves with O started on the first 1.57; P in a
// loop over TMEM instead of registers 1.58 (each against 1.52); S in two halves of
// 64 columns, the second beside P V^ 1.56 (against 1.46: an MMA of 64 columns reads
// as much of the queries as one of 128); one CTA per SM that works off an equal
// share of all tiles, with partials where a share ends inside a block, 1.57; the
// queries as bulk copies to V^'s place 1.45 (both against 1.43).
#include "kvq_block8.cuh"
#include "kvq_common.cuh"
#include "kvq_host.cuh"
#include "kvq_tc.cuh"

#include <type_traits>

namespace kvq {
namespace {

constexpr int kT = 128;         // cache positions per tile
constexpr int kRows = 128;      // rows of one query tile (the MMA's M)
constexpr int kXTiles = 2;      // query tiles per CTA
constexpr int kCtaRows8 = kXTiles * kRows;
constexpr int kSmWarps = 4 * kXTiles;
constexpr int kExpWarps = 4;
constexpr int kLdWarp = kSmWarps + kExpWarps;
constexpr int kMWarp = kLdWarp + 1;
constexpr int kScWarp = kMWarp + kXTiles;
// four warpgroups, so that registers can move between them: the loader's and
// the MMA issuers' group and the expansion leave theirs
// to the softmax, which holds a row's 128 scores at once
constexpr int kP8Threads = 512;
constexpr int kRegsSoftmax = 192, kRegsExpand = 72, kRegsIssue = 56;  // 2 x 192 + 72 + 56 = 4 x 128
static_assert(2 * kRegsSoftmax + kRegsExpand + kRegsIssue <= 4 * 128, "registers of the launch");
// TMEM: S_X, then P_X, at [128 X, +128), O_X at [256 + 128 X, +d).  (At head_dim
// 64 P_X fits beside S_X, and the next scores need not wait for the product that
// reads it; but there the softmax is the bound: 1% slower for a chunk of 1024 over
// 16384 positions, 4 x 64 heads.)
constexpr int kOCol8 = kXTiles * kT;
constexpr int kTmem8 = 512;
constexpr int kKRing = 3, kVRing = 3, kVSlots8 = 2;
// The running maximum is raised only when a score passes it by this much (log2):
// f16 holds 2^15, and among 32 rows with heavy-tailed scores a smaller slack has
// some row raise it on every few tiles (prefill of 1024 over 16384 positions,
// 4 x 64 heads: 8 1529 us, 12 1488, 15 1459).
constexpr float kSlack8 = 15.0f;
// log2 of P over 2^(y - m): from kMinFactor up in P, to kMaxFactor in l (where more
// makes the weight one under 2^-105).
constexpr float kMinFactor = -60.0f, kMaxFactor = 120.0f;
// m is raised when it is this far under a score beside a held exponent, and once l
// has grown to kMaxSum; between, l counts what m lags.
// Value scales that differ by this much (log2; f16 has 14 before its subnormals) give the
// tokens of a partly attended tile exponents of their own; V^ of such a token is under
// 2^(kTokenTop + 1).
constexpr uint32_t kScaleSpread = 10;
constexpr int kTokenTop = 5;
constexpr float kIntBias = 12582912.0f;  // 1.5 * 2^23: the sum's low bits are the integer
constexpr float kSlackSum = 4.0f, kMaxSum = 1073741824.0f;  // 2^30
constexpr uint32_t kPoll8 = 20000;
constexpr int kScaleBytes = 128;  // scales of one tile: up to 8 groups of 16 bytes

enum : int {
  kKFull = 0,                      // [kKRing] K codes and scales landed
  kKEmpty = kKFull + kKRing,       // [kKRing] S products done (commit), softmax warps have the scales
  kScFull = kKEmpty + kKRing,      // [2 kKRing] the tile's scales as the softmax takes them
  kV8Full = kScFull + 2 * kKRing,      // [kVRing] V codes and scales landed
  kV8Empty = kV8Full + kVRing,     // [kVRing] expanded (one arrival per warp)
  kVFull = kV8Empty + kVRing,      // [kVSlots8] V^ slot written
  kVEmpty = kVFull + kVSlots8,     // [kVSlots8] O products done with it (commit)
  kSFull = kVEmpty + kVSlots8,     // [kXTiles] S_X in TMEM
  kPFull = kSFull + kXTiles,       // [kXTiles] P_X in TMEM, O_X rescaled
  kPvDone = kPFull + kXTiles,      // [kXTiles] O_X += P_X V^ done
  kTurn = kPvDone + kXTiles,       // [kXTiles] query tile X's products may be issued
  kTok = kTurn + kXTiles,          // the expansion's threads have looked at a tile's tokens
  kBars8 = kTok + 1
};

struct Prefill8Params {
  const int32_t* lens;
  const int32_t* chunk_lens;
  kvq_cache c;
  const uint16_t* q;
  void* out;
  float* part_o;   // [parts][batch * chunk * hq][D] when parts > 1: a part's own result O / l
  float* part_ml;  // [parts][batch * chunk * hq][2]: its m and l
  int32_t* flag;
  int32_t batch, hkv, g, hq, chunk, splits, qpb, nqb, out_bf16;
  int32_t parts;   // partials per row: splits, or twice that for a pair
  uint32_t g_inv;  // 2^16 / g rounded up: row / g is row * g_inv >> 16 for rows < 512
  float qk_log2;
  uint64_t wait_ns;  // a test's limit of the waits, or 0
};

template <int D>
struct P8Geo {
  static constexpr int kQBytes = kRows * D;              // one tile of hi or lo
  static constexpr int kQ = 0;                           // [tile][hi, lo]
  static constexpr int kK = kQ + 2 * kXTiles * kQBytes;  // [kKRing][128 positions][D]
  static constexpr int kV8 = kK + kKRing * kT * D;       // [kVRing]
  static constexpr int kV = kV8 + kVRing * kT * D;       // [kVSlots8][D][128] f16
  static constexpr int kKS = kV + kVSlots8 * kT * D * 2;
  static constexpr int kVS = kKS + kKRing * kScaleBytes;
  // [2 kKRing][8] (sK, log2 sV), with kScFull and emin: a tile's are read by the softmax
  // until the tile one K ring later has been taken, and by the expansion until then too
  // (the tile before that one has its scores only once this tile's product is issued)
  static constexpr int kSc = kVS + kVRing * kScaleBytes;
  static constexpr int kTokExp = kSc + 2 * kKRing * 64;    // [kVSlots8][128] a token's exponent, biased
  static constexpr int kTokMul = kTokExp + kVSlots8 * kT;  // [128] a token's factor in V^, f16
  static constexpr int kNan = kTokMul + kT * 2;  // [D] per channel the first position (of the CTA's) whose value is NaN
  static constexpr int kBar = kNan + 4 * D;
  static constexpr int kMisc = kBar + 8 * kBars8;        // TMEM slot, abort, first NaN, masks, exponents, ends
  static constexpr int kMiscEnd = kMisc + 4 * (3 + 3 * kKRing + kVRing + 2 + 2 * kXTiles);
  // where a half's rows are turned for coalesced stores: 128 bytes a row.  At
  // head_dim 128 that is query memory that no product reads any more: the half's
  // own tile's, for a pair the second tile's, which holds no queries
  static constexpr int kStage = (kMiscEnd + 127) / 128 * 128;
  static constexpr int kStageBytes = 128 * kRows;
  static constexpr bool kStageInQ = kQBytes >= kStageBytes;
  static constexpr int kUsed = (kStageInQ ? kMiscEnd : kStage + kXTiles * kStageBytes) + 128;
  // at least half an SM's shared memory, so that one CTA (holding all 512
  // TMEM columns) runs per SM
  static constexpr int kBytes = kUsed > 116 * 1024 ? kUsed : 116 * 1024;
  static_assert(kBar % 8 == 0 && kBytes <= 227 * 1024, "shared-memory layout");
};

// A wait of the whole warp with one outcome (TMEM accesses are warp-collective); it
// gives up after the library's limit, or with any other wait of the CTA.  TEST: the
// instantiation with a test's limit, which polls (a suspending wait could outlast it).
template <bool TEST>
struct Waits {
  volatile int* abort;
  uint64_t limit;  // TEST, ns
  __device__ __forceinline__ bool look(uint32_t bar, uint32_t parity) const {
    return TEST ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
  }
  __device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity) const {
    if (look(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (true) {
      if (look(bar, parity)) return true;
      if (*abort) return false;
      if (global_ns() - t0 > (TEST ? limit : kWaitLimitNs)) {
        *abort = 1;
        return false;
      }
    }
  }
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xFFFFFFFFu, lane_wait(bar, parity));
  }
};

__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void upk2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// D[tmem] (+)= A[desc] * B[desc]^T, E4M3 operands, fp32 accumulator.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Scale pair of 16-position block i of a tile staged by groups of GT tokens.
template <int GT>
__device__ __forceinline__ uint32_t scale_at(uint32_t base, int i) {
  return base + (GT == 16 ? 16 * i : 8 * i);
}

// 16 columns of this warp's TMEM lanes and their maximum, without the wait.
__device__ __forceinline__ void tmem_ld_max16_async(uint32_t taddr, uint32_t (&v)[16], uint32_t& m) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, "
      "[%17];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(m)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld_all() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
// keeps the uses of v and m behind the wait
__device__ __forceinline__ void after_wait(uint32_t (&v)[16], uint32_t& m) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(m)
               :
               : "memory");
}

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}

// P = 2^(S csk + c) for the 16 scores of a block as 8 f16 pairs; their sum times
// f into l2.
__device__ __forceinline__ void block_p(const uint32_t (&v)[16], uint32_t* w, float csk, float c, float f,
                                        uint64_t& l2) {
  const uint64_t cs2 = pk2(csk, csk), c2 = pk2(c, c);
  uint64_t sum = 0ull;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float y0, y1;
    upk2(fma2(pk2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), cs2, c2), y0, y1);
    const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
    sum = i == 0 ? pk2(e0, e1) : add2(sum, pk2(e0, e1));
    w[i] = pack_f16x2(e0, e1);
  }
  l2 = fma2(sum, pk2(f, f), l2);
}

// The part of a V scale that goes into P's exponent: 2^e = its power of two, with
// e from -126 (fp32's subnormals keep the rest in the significand) to 120 (where
// the rest times a code stays an f16 value for every finite product).
__device__ __forceinline__ uint32_t v_exponent(uint32_t bits) { return min(max(bits >> 23, 1u), 247u); }
// e as a float, from v_exponent's biased form
__device__ __forceinline__ float v_log2(uint32_t e) { return __uint_as_float(0x4B000000u | e) - (8388608.0f + 127.0f); }
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
// the rest, sV / 2^e
__device__ __forceinline__ float v_rest(uint32_t bits) {
  return __uint_as_float(bits) * __uint_as_float((254u - v_exponent(bits)) << 23);
}

// A load that is issued where it stands.
__device__ __forceinline__ uint4 ldg128_now(const void* ptr) {
  uint4 r;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(ptr));
  return r;
}

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hsub2_u32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_from_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(v));
  return r;
}

// 8 columns of this warp's TMEM lanes, without the wait.
__device__ __forceinline__ void tmem_st8_async(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// PAIR: few rows: both halves of the CTA serve one query tile, every second cache
// tile each.
template <int D, int GT, bool PAIR, bool TEST>
__global__ void __launch_bounds__(kP8Threads, 1) prefill_block8_kernel(const Prefill8Params p) {
  using G = P8Geo<D>;
  // K slots in use.  A pair's half sees every second tile only: with two slots it
  // waits on the same barrier phase after phase.  (With three it would skip phases,
  // and could take a tile that is still on its way for the one before.)
  constexpr int kRing = PAIR ? 2 : kKRing;
  constexpr int kGroups = kT / GT;
  constexpr int kGroupBytes = 2 * GT * D + (GT >= 32 ? GT / 2 : 16);
  constexpr int kGroupScale = GT >= 32 ? GT / 2 : 16;
  extern __shared__ uint8_t p8_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p8_raw) + 127) & ~uintptr_t(127));
  const uint32_t sb = smem_addr(base);
  const uint32_t bars = sb + G::kBar;
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + G::kMisc);
  uint32_t* tslot = misc;
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 1);
  const Waits<TEST> wait{abort, p.wait_ns};
  volatile uint32_t* kgood = misc + 3;             // [kKRing] bit i: block i of the tile lies in a valid page
  volatile uint32_t* vgood = misc + 3 + kKRing;    // [kVRing]
  volatile uint32_t* emin = misc + 3 + kKRing + kVRing;  // [2 kKRing] the smallest log2 sV of the tile; NaN: its tokens have exponents of their own
  // what can still be on its way at the end: the loader's K and V tiles so far, and each
  // MMA warp's last commit (barrier and parity)
  volatile uint32_t* ends = misc + 3 + 3 * kKRing + kVRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int sp = (int)(blockIdx.x % (unsigned)p.splits);
  const int rest = (int)(blockIdx.x / (unsigned)p.splits);
  const int qb = p.nqb - 1 - rest % p.nqb;  // the longest first
  const int bh = rest / p.nqb;
  const int h = bh % p.hkv, b = bh / p.hkv;
  const int32_t T = __ldg(p.lens + b);
  // the query rows' loads, in flight while the lengths are looked at
  uint4 qv[4][D / 32];
#pragma unroll
  for (int rg = 0; rg < 4; ++rg) {
    const int qr = (PAIR ? warp & 3 : warp) * 32 + 8 * rg + (lane >> 2);
    const int qt = (int)((unsigned)qr * p.g_inv >> 16);  // qr / g
    const int qti = qb * p.qpb + qt;
    const bool in = warp < kSmWarps && qr < p.qpb * p.g && qti < p.chunk;
    const uint16_t* src = p.q + (((int64_t)b * p.chunk + qti) * p.hq + h * p.g + qr - qt * p.g) * D + (lane & 3) * 8;
#pragma unroll
    for (int cg = 0; cg < D / 32; ++cg) {
      qv[rg][cg] = make_uint4(0u, 0u, 0u, 0u);
      if (in) qv[rg][cg] = ldg128_now(src + 32 * cg);
    }
  }
  const int n = p.chunk_lens ? __ldg(p.chunk_lens + b) : p.chunk;
  if (n < 0 || n > p.chunk || T < 0) {
    if (tid == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
    if (n < 0 || n > p.chunk) return;
  }
  if (qb * p.qpb >= n) return;  // padding only
  const int X = tid / kRows;                   // softmax threads: the half of the CTA,
  const int r = PAIR ? tid % kRows : tid;    // the row,
  const int rt = (int)((unsigned)r * p.g_inv >> 16);  // r / g
  const int ti = qb * p.qpb + rt;              // its query token and head
  const int hh = h * p.g + r - rt * p.g;
  const bool row_ok = tid < kCtaRows8 && r < p.qpb * p.g && ti < n;
  const int part = PAIR ? 2 * sp + X : sp;   // which of the row's partials
  const int64_t row = ((int64_t)b * p.chunk + ti) * p.hq + hh;
  const int64_t rows_all = (int64_t)p.batch * p.chunk * p.hq;
  if (T < n) {  // the chunk's own tokens must be in the cache
    if (tid == 0) set_flag(p.flag, KVQ_FLAG_BAD_LENGTH);
    if (row_ok) {
      if (p.parts > 1) {
        *(reinterpret_cast<float2*>(p.part_ml) + part * rows_all + row) = make_float2(-INFINITY, 0.0f);
      } else {
        for (int c = 0; c < D; c += 8) {
          if (p.out_bf16) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + c) = make_uint4(0u, 0u, 0u, 0u);
          } else {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * D + c);
            o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
    }
    return;
  }
  const int64_t first = (int64_t)T - n;             // position of the chunk's token 0
  const int64_t pos_min = first + qb * p.qpb;       // last position that every row of the CTA attends
  const int last_ti = min(n, (qb + 1) * p.qpb) - 1;
  const int64_t cap = (int64_t)p.c.max_pages_per_seq * p.c.page_size;
  const int64_t limit = min(first + last_ti + 1, cap);  // positions read
  if (tid == 0 && first + last_ti + 1 > cap) set_flag(p.flag, KVQ_FLAG_PAGE_OOB);
  const int tiles = (int)((limit + kT - 1) / kT);
  const int per = (tiles + p.splits - 1) / p.splits;
  const int j0 = min(tiles, sp * per), ntiles = min(tiles, j0 + per) - j0;
  const int rows_used = (last_ti - qb * p.qpb + 1) * p.g;
  const int nx = PAIR ? min(2, ntiles) : rows_used > kRows ? 2 : 1;  // halves with work
  const int users = PAIR ? 1 : nx;                // halves that read one cache tile
  const int step = PAIR ? 2 : 1;
  if (ntiles <= 0) {                                // a split without positions
    if (row_ok) *(reinterpret_cast<float2*>(p.part_ml) + part * rows_all + row) = make_float2(-INFINITY, 0.0f);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kKRing; ++i) {
      mbar_init(bars + 8 * (kKFull + i), 1);
      mbar_init(bars + 8 * (kKEmpty + i), 5 * users);
      mbar_init(bars + 8 * (kScFull + i), 1);
      mbar_init(bars + 8 * (kScFull + kKRing + i), 1);
    }
    for (int i = 0; i < kVRing; ++i) {
      mbar_init(bars + 8 * (kV8Full + i), 1);
      mbar_init(bars + 8 * (kV8Empty + i), kExpWarps);
    }
    for (int i = 0; i < kVSlots8; ++i) {
      mbar_init(bars + 8 * (kVFull + i), 32 * kExpWarps);
      mbar_init(bars + 8 * (kVEmpty + i), users);
    }
    for (int i = 0; i < kXTiles; ++i) {
      mbar_init(bars + 8 * (kSFull + i), 1);
      mbar_init(bars + 8 * (kPFull + i), 4);
      mbar_init(bars + 8 * (kPvDone + i), 1);
      mbar_init(bars + 8 * (kTurn + i), 1);
    }
    mbar_init(bars + 8 * kTok, 32 * kExpWarps);
    *abort = 0;
    fence_barrier_init();
  }
  int* nan_first = reinterpret_cast<int*>(base + G::kNan);
  int* nan_least = reinterpret_cast<int*>(misc + 2);  // the smallest of them
  if (warp == 0) tmem_alloc(smem_addr(tslot), kTmem8);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tslot);

  const uint8_t* pool = static_cast<const uint8_t*>(p.c.data);
  const Block8Layout L(D, p.c.page_size);
  // The loader warp's copies of tile j: lane i < kGroups takes group i, K codes
  // and scales, then V codes and scales.  The lanes look up the groups of 32 /
  // kGroups tiles at once.
  int kiss = 0, viss = 0;  // tiles so far
  const uint8_t* src_l = nullptr;
  const auto load_tile = [&](int j) -> bool {
    const int ks = j % kRing, vs = j % kVRing;
    const int g_first = j % (32 / kGroups) * kGroups;
    if (g_first == 0) {
      const int64_t pos = (int64_t)(j0 + j) * kT + lane * GT;
      src_l = nullptr;
      if (pos < limit && pos < (int64_t)(j0 + ntiles) * kT) {
        const int64_t phys = block8_page(p.c, b, pos, p.flag);
        if (phys >= 0) {
          const int64_t off = block8_group_offset(L, phys, p.hkv, h, (int)(pos & (p.c.page_size - 1)));
          if (KVQ_IN(off >= 0 && off + kGroupBytes <= p.c.num_pages * (int64_t)p.hkv * L.page_bytes(), p.flag))
            src_l = pool + off;
        }
      }
    }
    const uint32_t got = (__ballot_sync(0xFFFFFFFFu, src_l != nullptr) >> g_first) & ((1u << kGroups) - 1u);
    const uint8_t* src = reinterpret_cast<const uint8_t*>(
        __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src_l), (g_first + lane) & 31));
    if (lane >= kGroups) src = nullptr;
    uint32_t good = 0u;
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
      if ((got >> i) & 1u) good |= ((1u << (GT / 16)) - 1u) << (i * (GT / 16));
    const uint32_t bytes = (uint32_t)__popc(got) * (uint32_t)(GT * D + kGroupScale);
    if (j >= kRing && !wait(bars + 8 * (kKEmpty + ks), (uint32_t)(j / kRing - 1) & 1u)) return false;
    if (lane == 0) {
      kgood[ks] = good;
      mbar_arrive_expect_tx(bars + 8 * (kKFull + ks), bytes);
    }
    __syncwarp();
    if (src != nullptr) {
      bulk_g2s(sb + G::kK + ks * kT * D + lane * GT * D, src, GT * D, bars + 8 * (kKFull + ks));
      bulk_g2s(sb + G::kKS + ks * kScaleBytes + lane * kGroupScale, src + 2 * GT * D, kGroupScale,
               bars + 8 * (kKFull + ks));
    }
    kiss = j + 1;
    if (j >= kVRing && !wait(bars + 8 * (kV8Empty + vs), (uint32_t)(j / kVRing - 1) & 1u)) return false;
    if (lane == 0) {
      vgood[vs] = good;
      mbar_arrive_expect_tx(bars + 8 * (kV8Full + vs), bytes);
    }
    __syncwarp();
    if (src != nullptr) {
      bulk_g2s(sb + G::kV8 + vs * kT * D + lane * GT * D, src + GT * D, GT * D, bars + 8 * (kV8Full + vs));
      bulk_g2s(sb + G::kVS + vs * kScaleBytes + lane * kGroupScale, src + 2 * GT * D, kGroupScale,
               bars + 8 * (kV8Full + vs));
    }
    viss = j + 1;
    return true;
  };
  if (warp < kSmWarps) {
    // query rows: power-of-two prescale, hi and lo E4M3 parts in operand layout.
    // Four lanes share a row's 16-byte parts (a thread per row would touch 32 lines
    // a load), and a warp's stores are whole core matrices.
    float cs;
    const uint32_t dst = sb + G::kQ + (PAIR ? 0 : X) * 2 * G::kQBytes + (uint32_t)((warp & 3) * 32 * D + (lane >> 2) * 16);
    uint32_t amax = 0u;  // of the thread's own row
    int k_own = 0;
    // (a loop, with the rows ahead moved down: the instructions of this part are
    // fetched for one pass only)
#pragma unroll 1
    for (int rg = 0; rg < 4; ++rg) {
      uint32_t am = 0u;
#pragma unroll
      for (int cg = 0; cg < D / 32; ++cg) {
        const uint32_t ws[4] = {qv[0][cg].x, qv[0][cg].y, qv[0][cg].z, qv[0][cg].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) am = max_u16x2(am, ws[i] & 0x7FFF7FFFu);
      }
      am = max(am << 16, am & 0xFFFF0000u);
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      int k = 0;
      if (am > 0u && am < 0x7F800000u) k = min(100, max(-120, 7 - ((int)(am >> 23) - 127)));
      const float up = __uint_as_float((uint32_t)(k + 127) << 23);
      if (!PAIR || X == rg >> 1) {  // (the halves of a pair prepare half of the rows each)
#pragma unroll
        for (int cg = 0; cg < D / 32; ++cg) {
          const uint32_t ws[4] = {qv[0][cg].x, qv[0][cg].y, qv[0][cg].z, qv[0][cg].w};
          uint32_t hp[4], lp[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // f16 holds the scaled values exactly down to 2^-17, where both parts are
            // zero, and their difference from hi
            const uint32_t x = pack_f16x2(bf16_lo(ws[i]) * up, bf16_hi(ws[i]) * up);
            hp[i] = e4m3x2_from_f16x2(x);
            lp[i] = e4m3x2_from_f16x2(hsub2_u32(x, f16x2_from_e4m3x2(hp[i])));
          }
          const uint32_t at = dst + (uint32_t)(rg * 8 * D + (2 * cg + ((lane & 3) >> 1)) * 128 + (lane & 1) * 8);
          sts64(at, hp[0] | (hp[1] << 16), hp[2] | (hp[3] << 16));
          sts64(at + G::kQBytes, lp[0] | (lp[1] << 16), lp[2] | (lp[3] << 16));
        }
      }
      const uint32_t am_r = __shfl_sync(0xFFFFFFFFu, am, (lane & 7) * 4);
      const int k_r = __shfl_sync(0xFFFFFFFFu, k, (lane & 7) * 4);
      if (lane >> 3 == rg) {
        amax = am_r;
        k_own = k_r;
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int cg = 0; cg < D / 32; ++cg) qv[i][cg] = qv[i + 1][cg];
    }
    cs = p.qk_log2 * __uint_as_float((uint32_t)(127 - k_own) << 23);
    if (amax >= 0x7F800000u) cs = __uint_as_float(0x7FC00000u);  // Inf or NaN query: the row is NaN
    fence_async_smem();
    asm volatile("bar.arrive 2, %0;\n" ::"r"(32 * (kSmWarps + nx)) : "memory");  // the MMA warps wait for the queries
    // ---------------------------------------------------------------- softmax
    reg_inc<kRegsSoftmax>();
    if (X >= nx) {  // a half without tiles
      if (PAIR && row_ok)
        *(reinterpret_cast<float2*>(p.part_ml) + part * rows_all + row) = make_float2(-INFINITY, 0.0f);
    } else {
      const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t sp_col = t_lane + (uint32_t)(X * kT);
      const uint32_t op = t_lane + (uint32_t)(kOCol8 + X * kT);
      const uint32_t s_full = bars + 8 * (kSFull + X), p_full = bars + 8 * (kPFull + X);
      const uint32_t pv_done = bars + 8 * (kPvDone + X);
      const int64_t pos_r = first + ti;  // last position this row attends
      float m_run = -INFINITY, mv_run = -INFINITY, l_run = 0.0f;  // m, m', l
      bool ok = true;
      uint32_t i_own = 0;  // this half's tiles so far
      // A block's exponent in P, beside y, and its factor in l, both from log2 sV and
      // the references.
      const auto factors = [&](const float (&lv)[8], float (&pc)[8], float (&pf)[8]) {
        const float mo = m_run == -INFINITY ? 0.0f : m_run;
        const float dm = mo - (mv_run == -INFINITY ? 0.0f : mv_run);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = fmaxf(lv[i] + dm, kMinFactor);
          pc[i] = a - mo;
          // 2^-a of a whole number, no less than 2^-kMaxFactor
          pf[i] = __uint_as_float(__float_as_uint(fmaxf(kIntBias + 127.0f - a, kIntBias + 127.0f - kMaxFactor)) << 23);
        }
      };
      // Lazy references: when m' is raised O shrinks (by al), when m is l does (al_l).
      // Returns whether a row of the warp raised m' (TMEM accesses are warp-collective).
      const auto raise = [&](float mt, float mv, float& al, float& al_l) -> bool {
        const bool up = mv > mv_run + kSlack8, any_up = __any_sync(0xFFFFFFFFu, up);
        if (up) {
          const float to = ceilf(mv);
          if (mv_run != -INFINITY) al = fast_exp2(mv_run - to);
          mv_run = to;
        }
        if (mt > m_run + kSlackSum) {
          const float to = ceilf(mt);
          if (m_run != -INFINITY) al_l = fast_exp2(m_run - to);
          m_run = to;
        }
        return any_up;
      };
      // P is on its way to TMEM: O_X rescaled, P handed over, l.
      const auto finish = [&](bool any_up, float al, float al_l, float sum) -> bool {
        if (any_up && i_own > 0) {
          if (!wait(pv_done, (i_own - 1) & 1u)) {
            tmem_wait_st();  // P's stores end before the TMEM does
            return false;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(op + (uint32_t)c0, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            tmem_st32_async(op + (uint32_t)c0, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        l_run = l_run * al_l + sum;
        if (l_run > kMaxSum) {
          const uint32_t k = min((__float_as_uint(l_run) >> 23) - 127u, 127u);
          l_run *= __uint_as_float((127u - k) << 23);
          m_run += (float)k;
        }
        return true;
      };
      // One cache tile; MASKED: some of its scores are not attended.  Two bodies, so
      // that the whole tiles' is one straight run of instructions.
      const auto tile = [&](auto masked_c, int j, uint32_t good, const float (&csk_in)[8], uint32_t sc,
                            float (&pc)[8], float (&pf)[8], bool held) -> bool {
        constexpr bool MASKED = decltype(masked_c)::value;
        float csk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) csk[i] = csk_in[i];
        if (!wait(s_full, i_own & 1u)) return false;
        tc_fence_after();
        // the row's 128 scores in registers, each block's maximum with them
        uint32_t v[8][16], vm[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) tmem_ld_max16_async(sp_col + (uint32_t)(16 * i), v[i], vm[i]);
        tmem_wait_ld_all();
#pragma unroll
        for (int i = 0; i < 8; ++i) after_wait(v[i], vm[i]);
        if constexpr (MASKED) {
          const int64_t p0 = (int64_t)(j0 + j) * kT;
          const int lim = row_ok ? (int)min((int64_t)kT, max((int64_t)0, pos_r - p0 + 1)) : 0;
          // masked scores (behind the row's last position, or in a page that is
          // not valid) become -inf, their factor positive: 2^-inf is 0
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int left = ((good >> i) & 1u) ? lim - 16 * i : 0;
            float a = -INFINITY;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              v[i][c] = c < left ? v[i][c] : 0xFF800000u;
              a = fmaxf(a, __uint_as_float(v[i][c]));
            }
            vm[i] = __float_as_uint(a);
            if (left < 16) csk[i] = left > 0 ? fmaxf(csk[i], 1e-37f) : 1.0f;
            if (cs != cs) csk[i] = cs;
          }
        }
        float y[8];  // y + log2 sV - m'
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(__uint_as_float(vm[i]), csk[i], pc[i]);
        const float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
        float al = 1.0f, al_l = 1.0f;
        bool any_up = false;
        if (__any_sync(0xFFFFFFFFu, top > (mv_run == -INFINITY ? -INFINITY : kSlack8)) || held) {
          float mt = -INFINITY, mv = -INFINITY, lv[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = __uint_as_float(vm[i]) * csk[i];
            lv[i] = __uint_as_float(lds32(sc + 8 * i + 4));
            mt = fmaxf(mt, x);
            mv = fmaxf(mv, x + lv[i]);
          }
          any_up = raise(mt, mv, al, al_l);
          factors(lv, pc, pf);
        }
        uint64_t l2[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint32_t w[16];
          block_p(v[i], w, csk[i], pc[i], pf[i], l2[0]);
          block_p(v[i + 1], w + 8, csk[i + 1], pc[i + 1], pf[i + 1], l2[1]);
          tmem_st16_async(sp_col + (uint32_t)(8 * i), w);
        }
        float a0, a1, b0, b1;
        upk2(l2[0], a0, a1);
        upk2(l2[1], b0, b1);
        return finish(any_up, al, al_l, (a0 + a1) + (b0 + b1));
      };
      // A tile whose tokens have exponents of their own: 16 scores at a time, from TMEM
      // once for the references and once for P (whose columns are those of scores that
      // have been taken).
      const auto tile_tokens = [&](int j, uint32_t good, uint32_t sc) -> bool {
        if (!wait(s_full, i_own & 1u)) return false;
        tc_fence_after();
        // The tokens' exponents come with V^.  Behind the scores: they follow this half's
        // last product, so the slot's phase before this tile's is over (ahead of them a
        // pair's half could find the barrier a whole phase behind, and pass).
        if (!wait(bars + 8 * (kVFull + j % kVSlots8), (uint32_t)(j / kVSlots8) & 1u)) return false;
        const int64_t p0 = (int64_t)(j0 + j) * kT;
        const int lim = row_ok ? (int)min((int64_t)kT, max((int64_t)0, pos_r - p0 + 1)) : 0;
        const uint32_t tok = sb + G::kTokExp + (uint32_t)(j % kVSlots8 * kT);
        // block i: its y (-inf where not attended), and its tokens' exponents, four in a word
        const auto take = [&](int i, float (&y)[16], uint32_t (&e)[4]) {
          uint32_t v[16];
          tmem_ld16(sp_col + (uint32_t)(16 * i), v);
          const float ck = cs * __uint_as_float(lds32(sc + (uint32_t)(8 * i)));
          const int left = ((good >> i) & 1u) ? lim - 16 * i : 0;
#pragma unroll
          for (int c = 0; c < 16; ++c) y[c] = c < left ? __uint_as_float(v[c]) * ck : -INFINITY;
          const uint4 x = lds128(tok + (uint32_t)(16 * i));
          e[0] = x.x, e[1] = x.y, e[2] = x.z, e[3] = x.w;
        };
        const auto exponent = [](const uint32_t (&e)[4], int c) { return __byte_perm(e[c >> 2], 0u, 0x4440u + (uint32_t)(c & 3)); };
        float y[16], mt = -INFINITY, mv = -INFINITY, sum = 0.0f;
        uint32_t e[4];
#pragma unroll 1
        for (int i = 0; i < kT / 16; ++i) {
          take(i, y, e);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            mt = fmaxf(mt, y[c]);
            mv = fmaxf(mv, y[c] + v_log2(exponent(e, c)));
          }
        }
        float al = 1.0f, al_l = 1.0f;
        const bool any_up = raise(mt, mv, al, al_l);
        const float mo = m_run == -INFINITY ? 0.0f : m_run;
        const float r = fast_exp2(fminf(mo - (mv_run == -INFINITY ? 0.0f : mv_run), 126.0f));  // 2^(m - m')
#pragma unroll 1
        for (int i = 0; i < kT / 16; ++i) {
          uint32_t w[8];
          take(i, y, e);
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const float p0 = fast_exp2(y[c] - mo), p1 = fast_exp2(y[c + 1] - mo);
            sum += p0 + p1;
            // the token's 2^exponent over 2^m'; finite, as p can be 0
            const float f0 = fminf(__uint_as_float(exponent(e, c) << 23) * r, 3e38f);
            const float f1 = fminf(__uint_as_float(exponent(e, c + 1) << 23) * r, 3e38f);
            w[c / 2] = pack_f16x2(p0 * f0, p1 * f1);
          }
          tmem_st8_async(sp_col + (uint32_t)(8 * i), w);
        }
        return finish(any_up, al, al_l, sum);
      };
      for (int j = PAIR ? X : 0; j < ntiles; j += step, ++i_own) {
        // the tile's scales, ahead of its scores
        const int ks = j % kRing;
        const int is = j % (2 * kRing);
        if (!(ok = wait(bars + 8 * (kScFull + is), (uint32_t)(j / (2 * kRing)) & 1u))) break;
        const uint32_t sc = sb + G::kSc + is * 64;
        float csk[8], lv[8], pc[8], pf[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint4 x = lds128(sc + 8 * i);
          csk[i] = cs * __uint_as_float(x.x);
          lv[i] = __uint_as_float(x.y);
          csk[i + 1] = cs * __uint_as_float(x.z);
          lv[i + 1] = __uint_as_float(x.w);
        }
        factors(lv, pc, pf);
        const uint32_t good = kgood[ks];
        // some block's exponent is held at kMinFactor in some row
        const float least = __uint_as_float(emin[is]);
        const bool held = __any_sync(0xFFFFFFFFu, least + m_run < mv_run + kMinFactor);
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (kKEmpty + ks));
        const int64_t p0 = (int64_t)(j0 + j) * kT;
        const bool fast = p0 + kT - 1 <= pos_min && good == 0xFFu;
        if (fast) {
          ok = tile(std::false_type{}, j, good, csk, sc, pc, pf, held);
        } else if (__builtin_expect(least == least, 1)) {
          ok = tile(std::true_type{}, j, good, csk, sc, pc, pf, held);
        } else {
          ok = tile_tokens(j, good, sc);
        }
        if (!ok) break;
      }
      // the result once the last O_X += P_X V^ is done
      if (ok) ok = wait(pv_done, (i_own - 1) & 1u);
      if (ok) {
        tc_fence_after();
        const bool partial = p.parts > 1;
        // O's scale over l, in two factors: 2^(m' - m) alone can pass fp32's exponents
        const float f0 = m_run == -INFINITY ? 1.0f : fast_exp2(0.5f * (mv_run - m_run));
        const float f = f0 * (l_run > 0.0f || l_run != l_run ? 1.0f / l_run : 0.0f);
        if (partial && row_ok)
          *(reinterpret_cast<float2*>(p.part_ml) + part * rows_all + row) = make_float2(m_run, l_run);
        // 128 bytes of every row at a time, turned in shared memory so that eight
        // lanes store one row's (a thread per row would touch 32 lines a store)
        const bool bf = p.out_bf16 && !partial;
        const int64_t row0 = ((int64_t)b * p.chunk + qb * p.qpb) * p.hq + h * p.g;
        const int rel_own = row_ok ? (int)(row - row0) : -1;
        int rel[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rel[i] = __shfl_sync(0xFFFFFFFFu, rel_own, 4 * i + (lane >> 3));
        const uint32_t stage =
            sb + (G::kStageInQ ? G::kQ + (PAIR ? 1 : X) * 2 * G::kQBytes : G::kStage) + X * G::kStageBytes +
            (uint32_t)((warp & 3) * 32 * 128);
        const uint32_t st_w = stage + (uint32_t)(lane * 128);
        uint8_t* ob = partial ? reinterpret_cast<uint8_t*>(p.part_o + (part * rows_all + row0) * D)
                              : static_cast<uint8_t*>(p.out) + row0 * D * (bf ? 2 : 4);
        const int row_b = D * (bf ? 2 : 4);
        // NaN values that the row has seen and V^ has not (noted before the expansion that
        // this half's last product waited for)
        const int seen_to = row_ok ? (int)min(pos_r - (int64_t)j0 * kT, (int64_t)INT32_MAX - 1) : -1;
        const bool nans = __any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(nan_least) <= seen_to);
#pragma unroll 1
        for (int c0 = 0; c0 < row_b; c0 += 128) {
          if (bf) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t o[32];
              tmem_ld32(op + (uint32_t)(c0 / 2 + 32 * half), o);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = bf16x2_of(__uint_as_float(o[8 * i + 2 * k]) * f0 * f, __uint_as_float(o[8 * i + 2 * k + 1]) * f0 * f);
                sts128(st_w + (uint32_t)(((4 * half + i) ^ (lane & 7)) * 16), make_uint4(w[0], w[1], w[2], w[3]));
              }
            }
          } else {
            uint32_t o[32];
            tmem_ld32(op + (uint32_t)(c0 / 4), o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(__uint_as_float(o[4 * i + k]) * f0 * f);
              sts128(st_w + (uint32_t)((i ^ (lane & 7)) * 16), make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          if (__builtin_expect(nans, 0)) {  // into the thread's own row
            const int size = bf ? 2 : 4;
#pragma unroll 1
            for (int i = 0; i < 128; i += size) {
              const uint32_t at = st_w + (uint32_t)((((i >> 4) ^ (lane & 7)) << 4) + (i & 15));
              if (*reinterpret_cast<volatile int*>(nan_first + (c0 + i) / size) > seen_to) continue;
              sts16(at + (uint32_t)size - 2u, 0x7FC0u);  // the upper half of an fp32 NaN, or a bf16 one
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3);
            const uint4 w = lds128(stage + (uint32_t)(rr * 128 + (((lane & 7) ^ (rr & 7)) * 16)));
            if (rel[i] >= 0) *reinterpret_cast<uint4*>(ob + (int64_t)rel[i] * row_b + c0 + (lane & 7) * 16) = w;
          }
          __syncwarp();
        }
      }
    }
  } else if (warp < kSmWarps + kExpWarps) {
    // ------------------------------------------------------------ V expansion
    // item (channel c, 16-position block): one 16-byte row of codes to two
    // 16-byte rows of f16; lanes take consecutive channels, so loads and
    // stores touch 128 contiguous bytes per eight lanes
    reg_dec<kRegsExpand>();
    const int dt = tid - 32 * kSmWarps;
    // (ahead of the CTA's barrier, behind the queries' loads, these stores cost 4%)
    if (dt < D) nan_first[dt] = INT32_MAX;
    if (dt == 0) *nan_least = INT32_MAX;
    asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kExpWarps) : "memory");
    uint32_t looked = 0;  // phases of kTok
    for (int j = 0; j < ntiles; ++j) {
      const int s = j % kVRing, slot = j % kVSlots8;
      const uint32_t codes = sb + G::kV8 + s * kT * D, dst = sb + G::kV + slot * kT * D * 2;
      const int valid = (int)min((int64_t)kT, limit - (int64_t)(j0 + j) * kT);
      if (!wait(bars + 8 * (kV8Full + s), (uint32_t)(j / kVRing) & 1u)) break;
      if (j >= kVSlots8 && !wait(bars + 8 * (kVEmpty + slot), (uint32_t)(j / kVSlots8 - 1) & 1u)) break;
      const uint32_t good = vgood[s];
      const bool whole = valid == kT && good == 0xFFu;
      const uint32_t c = dt % D;
#pragma unroll 1
      for (int blk = dt / D; blk < kT / 16; blk += 32 * kExpWarps / D) {
        uint4 w = lds128(codes + ((uint32_t)(blk * D) + c) * 16);
        const float r = v_rest(lds32(scale_at<GT>(sb + G::kVS + s * kScaleBytes, blk) + 4));
        uint32_t r2 = pack_f16x2(r, r);
        uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        if (!whole) {  // positions that are not attended: zero codes and a finite factor
          const int left = ((good >> blk) & 1u) ? valid - 16 * blk : 0;
          if (left <= 0) r2 = 0u;
#pragma unroll
          for (int t = 0; t < 4; ++t)
            ws[t] &= (2 * t < left ? 0x000000FFu : 0u) | (2 * t + 1 < left ? 0x0000FF00u : 0u) |
                     (2 * t + 8 < left ? 0x00FF0000u : 0u) | (2 * t + 9 < left ? 0xFF000000u : 0u);
        }
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          lo[t] = hmul2_u32(f16x2_from_e4m3x2(ws[t] & 0xFFFFu), r2);
          hi[t] = hmul2_u32(f16x2_from_e4m3x2(ws[t] >> 16), r2);
        }
        const uint32_t at = dst + core_offset(c, (uint32_t)(16 * blk), D);
        sts128(at, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        sts128(at + (D / 8) * 128, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      }
      if (__builtin_expect((int64_t)(j0 + j) * kT + kT - 1 > pos_min, 0)) {  // some row sees it in part
        uint32_t nan = 0u;  // bit 7 of a byte: the code is NaN's, 0x7F or 0xFF
#pragma unroll
        for (int i = 0; i < kT / 16 * D / (32 * kExpWarps); ++i) {
          const uint4 w = lds128(codes + ((uint32_t)((dt / D + i * (32 * kExpWarps / D)) * D) + c) * 16);
          nan |= ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
                 ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
        }
        if (__builtin_expect((nan & 0x80808080u) != 0u, 0)) {
#pragma unroll 1
          for (int t = 0; t < valid; ++t) {
            const int blk = t >> 4;
            if (((good >> blk) & 1u) == 0u || blk % (32 * kExpWarps / D) != dt / D) continue;  // not the thread's item
            const uint32_t x = lds8(codes + ((uint32_t)(blk * D) + c) * 16 + (uint32_t)block8_v_byte(t & 15));
            if ((x & 0x7Fu) != 0x7Fu) continue;
            sts16(dst + core_offset(c, (uint32_t)t, D), 0u);
            atomicMin(nan_first + c, j * kT + t);
            atomicMin(nan_least, j * kT + t);
          }
        }
        const int is = j % (2 * kRing);
        if (!wait(bars + 8 * (kScFull + is), (uint32_t)(j / (2 * kRing)) & 1u)) break;
        if (emin[is] == 0x7FC00000u) {  // the tokens have exponents of their own
          // thread = token: its largest code
          const int blk = dt >> 4;
          const uint32_t row0 = codes + (uint32_t)(blk * D * 16 + block8_v_byte(dt & 15));
          uint32_t top = 0u;
#pragma unroll 4
          for (int k = 0; k < D; ++k) {
            const uint32_t x = lds8(row0 + 16u * (uint32_t)k) & 0x7Fu;
            top = max(top, x == 0x7Fu ? 0u : x);
          }
          const uint32_t e = v_exponent(lds32(scale_at<GT>(sb + G::kVS + s * kScaleBytes, blk) + 4));
          const int k = (int)(__float_as_uint(e4m3_to_f32(top)) >> 23) - 127;  // 2^k <= top < 2^(k+1)
          const bool zero = top == 0u || !((good >> blk) & 1u) || dt >= valid;
          // 2^up into V^: none where sV is next to fp32's smallest, or its largest with a rest of more than 2
          const int up = zero || e == 247u ? 0 : min(kTokenTop - k, (int)e - 1);
          sts8(sb + G::kTokExp + (uint32_t)(slot * kT + dt), zero ? 1u : e - (uint32_t)up);
          sts16(sb + G::kTokMul + (uint32_t)(2 * dt), (uint32_t)(up + 15) << 10);
          mbar_arrive(bars + 8 * kTok);
          if (!wait(bars + 8 * kTok, looked++ & 1u)) break;
#pragma unroll 1
          for (int t0 = 16 * (dt / D); t0 < kT; t0 += 16 * (32 * kExpWarps / D)) {  // the thread's own items
#pragma unroll
            for (int t = t0; t < t0 + 16; t += 8) {
              const uint32_t at = dst + core_offset(c, (uint32_t)t, D);
              const uint4 v = lds128(at), m = lds128(sb + G::kTokMul + (uint32_t)(2 * t));
              sts128(at, make_uint4(hmul2_u32(v.x, m.x), hmul2_u32(v.y, m.y), hmul2_u32(v.z, m.z), hmul2_u32(v.w, m.w)));
            }
          }
          // (one array of factors: every thread is done with it before the next such tile)
          mbar_arrive(bars + 8 * kTok);
          if (!wait(bars + 8 * kTok, looked++ & 1u)) break;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (kV8Empty + s));
      fence_async_smem();
      mbar_arrive(bars + 8 * (kVFull + slot));
    }
  } else {
   reg_dec<kRegsIssue>();
   if (warp == kLdWarp) {
    // ------------------------------------------------------------ bulk copies
    for (int j = 0; j < ntiles; ++j)
      if (!load_tile(j)) break;
    if (lane == 0) {
      ends[0] = (uint32_t)kiss;
      ends[1] = (uint32_t)viss;
    }
   } else if (warp == kScWarp) {
    // ------------------------------------------------------------ scales
    // what every row's softmax needs of the tile's 8 blocks: sK and log2 of sV's power
    // of two (once here instead of in 256 rows)
    uint32_t least = 255u;  // the smallest exponent so far
    for (int j = 0; j < ntiles; ++j) {
      const int ks = j % kRing, is = j % (2 * kRing);
      if (!wait(bars + 8 * (kKFull + ks), (uint32_t)(j / kRing) & 1u)) break;
      const uint2 sc = lds64(scale_at<GT>(sb + G::kKS + ks * kScaleBytes, lane & 7));
      const uint32_t e = v_exponent(sc.y), here = __reduce_min_sync(0xFFFFFFFFu, e);
      // (a scale of 2^-126 and less is that of zeros)
      const int64_t p0 = (int64_t)(j0 + j) * kT;
      const bool counts = ((kgood[ks] >> (lane & 7)) & 1u) && p0 + 16 * (lane & 7) < limit && e > 1u;
      least = min(least, __reduce_min_sync(0xFFFFFFFFu, counts ? e : 255u));
      const bool tokens =
          __reduce_max_sync(0xFFFFFFFFu, counts ? e : 0u) > least + kScaleSpread && p0 + kT - 1 > pos_min;
      if (lane < 8) sts64(sb + G::kSc + is * 64 + 8 * lane, sc.x, __float_as_uint(v_log2(e)));
      if (lane == 0) emin[is] = tokens ? 0x7FC00000u : __float_as_uint(v_log2(here));
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (kScFull + is));
    }
   } else if (warp - kMWarp < nx) {
    // ----------------------------------------------------------- tensor cores
    // One warp per query tile, each with the chain S(0), O(0), S(1), O(1) ..
    // of its own tile: a wait drains what its warp has issued, and the other
    // warp's products fill the tensor pipe meanwhile.  The whole warp walks the
    // tiles, so that descriptors and addresses stay in uniform registers; one
    // elected lane issues.
    constexpr uint32_t kIdS = idesc_f16_f32(kRows, kT);  // E4M3 is type 0 of kind::f8f6f4, as f16 is of kind::f16
    constexpr uint32_t kIdO = idesc_f16_f32(kRows, D);
    const int x = warp - kMWarp;
    const uint64_t dq = smem_desc(sb + G::kQ + (PAIR ? 0 : x) * 2 * G::kQBytes, 128, 8 * D);
    const uint64_t dk0 = smem_desc(sb + G::kK, 128, 8 * D);
    const uint64_t dv0 = smem_desc(sb + G::kV, (D / 8) * 128, 128);
    const uint32_t s_col = tmem + (uint32_t)(x * kT), o_col = tmem + (uint32_t)(kOCol8 + x * kT);
    const uint32_t s_full = bars + 8 * (kSFull + x), p_full = bars + 8 * (kPFull + x);
    const uint32_t pv_done = bars + 8 * (kPvDone + x);
    const auto issue_s = [&](int ring) {
      const uint64_t dk = dk0 + (uint64_t)(ring * (kT * D / 16));
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < D / 32; ++s) tc_mma_f8(s_col, dq + (uint64_t)(16 * s), dk + (uint64_t)(16 * s), kIdS, s > 0);
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
          tc_mma_f8(s_col, dq + (uint64_t)(G::kQBytes / 16 + 16 * s), dk + (uint64_t)(16 * s), kIdS, true);
        tc_commit(s_full);
        tc_commit(bars + 8 * (kKEmpty + ring));
      }
      __syncwarp();
    };
    uint32_t last_bar = 0, last_par = 0;  // the last commit
    int j = PAIR ? x : 0;              // this half's first tile (x < nx <= ntiles for a pair)
    asm volatile("bar.sync 2, %0;\n" ::"r"(32 * (kSmWarps + nx)) : "memory");  // the queries are written
    bool ok = wait(bars + 8 * (kKFull + j), 0u);
    if (ok) {
      tc_fence_after();
      issue_s(j);
      last_bar = s_full;
    }
    const bool turns = !PAIR && nx > 1;
    for (uint32_t i = 0; j < ntiles && ok; j += step, ++i) {
      const int jn = j + step, kr = jn % kRing, vslot = j % kVSlots8;
      const bool more = jn < ntiles;
      if (more && !(ok = wait(bars + 8 * (kKFull + kr), (uint32_t)(jn / kRing) & 1u))) break;
      if (!(ok = wait(bars + 8 * (kVFull + vslot), (uint32_t)(j / kVSlots8) & 1u))) break;
      if (!(ok = wait(p_full, i & 1u))) break;
      // A(0), B(0), A(1), ..: the tiles take turns, so that one's softmax runs
      // beside the other's products
      if (turns && (x > 0 || i > 0) && !(ok = wait(bars + 8 * (kTurn + x), (x > 0 ? i : i - 1) & 1u))) break;
      tc_fence_after();
      const uint64_t dv = dv0 + (uint64_t)(vslot * (kT * D * 2 / 16));
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < kT / 16; ++s)
          tc_mma_f16_ta(o_col, s_col + (uint32_t)(s * 8), dv + (uint64_t)(s * 2 * (D / 8) * 8), kIdO, i > 0 || s > 0);
        tc_commit(pv_done);
        tc_commit(bars + 8 * (kVEmpty + vslot));
      }
      __syncwarp();
      last_bar = pv_done;
      last_par = i & 1u;
      if (more) {
        // P lives in S's columns: the next scores follow the product that reads it
        if (!(ok = wait(pv_done, i & 1u))) break;
        tc_fence_after();
        issue_s(kr);
        last_bar = s_full;
        last_par = (i + 1) & 1u;
      }
      if (turns && lane == 0) mbar_arrive(bars + 8 * (kTurn + (x ^ 1)));
    }
    if (lane == 0) {
      ends[2 + 2 * x] = last_bar;
      ends[3 + 2 * x] = last_par;
    }
   }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // A wait gave up (every role is past its last one here, so the word is final): copies
  // and products still on their way land before shared memory and TMEM go away.
  if (*abort) {
    const auto land = [&](uint32_t bar, uint32_t parity) {
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait_hint(bar, parity, kPoll8) && global_ns() - t0 < 20000000ull) {
      }
    };
    if (warp == kLdWarp) {
      const int k = (int)ends[0], v = (int)ends[1];
      for (int j = max(0, k - kRing); j < k; ++j) land(bars + 8 * (kKFull + j % kRing), (uint32_t)(j / kRing) & 1u);
      for (int j = max(0, v - kVRing); j < v; ++j) land(bars + 8 * (kV8Full + j % kVRing), (uint32_t)(j / kVRing) & 1u);
    } else if (warp >= kMWarp && warp - kMWarp < nx && ends[2 + 2 * (warp - kMWarp)] != 0u) {
      land(ends[2 + 2 * (warp - kMWarp)], ends[3 + 2 * (warp - kMWarp)]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) set_flag(p.flag, KVQ_FLAG_TIMEOUT);
  }
  if (warp == 0) tmem_dealloc(tmem, kTmem8);
}

// Joins the splits' partials of one query row per D/4 threads.
template <int D>
__global__ void __launch_bounds__(256) prefill_merge_kernel(const Prefill8Params p) {
  grid_dependency_wait();
  const int64_t rows = (int64_t)p.batch * p.chunk * p.hq;
  const int64_t i = (int64_t)blockIdx.x * (256 / (D / 4)) + threadIdx.x / (D / 4);
  const int c4 = threadIdx.x % (D / 4);
  if (i >= rows) return;
  const int64_t tok = i / p.hq;
  const int b = (int)(tok / p.chunk), ti = (int)(tok % p.chunk);
  const int n = p.chunk_lens ? __ldg(p.chunk_lens + b) : p.chunk;
  if (n < 0 || n > p.chunk || ti >= n) return;
  // twelve partials at a time, their loads in flight together
  constexpr int kBatch = 12;
  float mx = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < p.parts; s0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t at = (int64_t)min(s0 + k, p.parts - 1) * rows + i;
      ml[k] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at);
      x[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + c4);
    }
    float mn = mx;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (s0 + k >= p.parts) ml[k] = make_float2(-INFINITY, 0.0f);
      mn = fmaxf(mn, ml[k].x);
    }
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float a = mx == -INFINITY ? 1.0f : fast_exp2(mx - ref);
    o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
    l *= a;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (ml[k].x == -INFINITY && ml[k].y == 0.0f) continue;  // no position of this row (its sums were not written)
      const float f = (ml[k].x == -INFINITY ? 1.0f : fast_exp2(ml[k].x - ref)) * ml[k].y;
      o = make_float4(fmaf(f, x[k].x, o.x), fmaf(f, x[k].y, o.y), fmaf(f, x[k].z, o.z), fmaf(f, x[k].w, o.w));
      l += f;
    }
    mx = mn;
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (p.out_bf16)
    *(reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + i * D) + c4) =
        make_uint2(bf16x2_of(o.x, o.y), bf16x2_of(o.z, o.w));
  else
    *(reinterpret_cast<float4*>(static_cast<float*>(p.out) + i * D) + c4) = o;
}

// ------------------------------------------------------------------ host side
constexpr int kMaxSplits = 32;

// CTAs that share the positions of one block of query rows: as many as keep
// the whole grid within one CTA per SM.
int prefill_splits(int64_t ctas, int sms) {
  const int64_t s = sms / (ctas > 0 ? ctas : 1);
  return (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

// The chunk's rows of one kv head fit one query tile: a CTA's two halves then
// share it and take every second cache tile each (a draft of 5 tokens x 8 heads
// over 9000 to 12345 positions, 2 sequences: 25.2 us against 28.6).
bool one_tile(int32_t chunk, int g) { return (int64_t)chunk * g <= kRows; }

size_t part_bytes(int64_t parts, int64_t rows, int d) {
  return parts > 1 ? (size_t)parts * (size_t)rows * (size_t)(d + 2) * sizeof(float) : 16;
}

template <int D, int GT, bool PAIR, bool TEST>
kvq_status launch_prefill8(const Prefill8Params& pp, cudaStream_t s, unsigned grid) {
  static DeviceOnce attr_set;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
  if (attr_set.pending(dev)) {
    if (cudaFuncSetAttribute(prefill_block8_kernel<D, GT, PAIR, TEST>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             P8Geo<D>::kBytes) != cudaSuccess)
      return KVQ_ERR_CUDA;
    attr_set.mark(dev);
  }
  prefill_block8_kernel<D, GT, PAIR, TEST><<<grid, kP8Threads, P8Geo<D>::kBytes, s>>>(pp);
  const kvq_status st = launch_status();
  if (st != KVQ_OK || pp.parts == 1) return st;
  const int64_t rows = (int64_t)pp.batch * pp.chunk * pp.hq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + 256 / (D / 4) - 1) / (256 / (D / 4))));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_merge_kernel<D>, pp) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

template <int D, bool PAIR>
kvq_status launch_prefill8_d(const Prefill8Params& pp, cudaStream_t s, unsigned grid) {
  switch (pp.c.page_size) {
    case 16: return launch_prefill8<D, 16, PAIR, false>(pp, s, grid);
    case 32: return launch_prefill8<D, 32, PAIR, false>(pp, s, grid);
    default: break;
  }
  return pp.wait_ns == 0 ? launch_prefill8<D, 64, PAIR, false>(pp, s, grid) : launch_prefill8<D, 64, PAIR, true>(pp, s, grid);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_fp8_block_prefill_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                                        int32_t head_dim, int32_t chunk) {
  if (batch < 1 || chunk < 1 || num_kv_heads < 1 || num_q_heads < num_kv_heads || num_q_heads % num_kv_heads != 0 ||
      num_q_heads / num_kv_heads > kCtaRows8 || head_dim < 16)
    return 0;
  const int sms = device_sm_count();
  if (sms <= 0) return 0;
  const int qpb = kCtaRows8 / (num_q_heads / num_kv_heads);
  const int64_t ctas = ((int64_t)chunk + qpb - 1) / qpb * batch * num_kv_heads;
  const int pair = one_tile(chunk, num_q_heads / num_kv_heads) ? 2 : 1;
  return part_bytes((int64_t)pair * prefill_splits(ctas, sms), (int64_t)batch * chunk * num_q_heads, head_dim);
}

extern "C" kvq_status kvq_fp8_block_prefill_attn(const kvq_cache* cache, int32_t batch, int32_t num_q_heads,
                                                 int32_t chunk, const int32_t* d_seq_lens, const int32_t* d_chunk_lens,
                                                 const void* q, float softmax_scale, void* out, int32_t out_dtype,
                                                 void* workspace, size_t workspace_bytes, int32_t* d_err_flag,
                                                 kvq_stream stream) {
  if (batch < 1 || chunk < 1) return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_status st = check_block8_cache(cache, batch);
  if (st != KVQ_OK) return st;
  const int hkv = cache->num_kv_heads, D = cache->head_dim;
  if (num_q_heads < hkv || num_q_heads % hkv != 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (!(softmax_scale > 0.0f) || !(softmax_scale < 3.0e38f)) return KVQ_ERR_INVALID_ARGUMENT;
  if (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16) return KVQ_ERR_INVALID_ARGUMENT;
  if (d_seq_lens == nullptr || q == nullptr || out == nullptr || workspace == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(workspace, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  const int g = num_q_heads / hkv;
  if (g > 8) return KVQ_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const int qpb = kCtaRows8 / g;
  const int64_t nqb = ((int64_t)chunk + qpb - 1) / qpb;
  const int64_t ctas = nqb * batch * hkv;
  if (ctas > 0x7FFFFFFF) return KVQ_ERR_UNSUPPORTED;
  // never more splits than the cache has tiles
  const int64_t cap_tiles = ((int64_t)cache->max_pages_per_seq * cache->page_size + kT - 1) / kT;
  int splits = prefill_splits(ctas, sms);
  const int64_t rows = (int64_t)batch * chunk * num_q_heads;
  const bool pair = one_tile(chunk, g);
  if (workspace_bytes < part_bytes((pair ? 2 : 1) * (int64_t)splits, rows, D)) return KVQ_ERR_WORKSPACE;
  if (splits > cap_tiles) splits = (int)cap_tiles;
  Prefill8Params pp = {};
  pp.lens = d_seq_lens;
  pp.chunk_lens = d_chunk_lens;
  pp.c = *cache;
  pp.q = static_cast<const uint16_t*>(q);
  pp.out = out;
  pp.part_o = static_cast<float*>(workspace);
  pp.parts = splits * (pair ? 2 : 1);
  pp.part_ml = pp.part_o + (size_t)pp.parts * rows * D;
  pp.flag = d_err_flag;
  pp.batch = batch;
  pp.hkv = hkv;
  pp.g = g;
  pp.g_inv = (65536u + (unsigned)g - 1) / (unsigned)g;
  pp.hq = num_q_heads;
  pp.chunk = chunk;
  pp.splits = splits;
  pp.qpb = qpb;
  pp.nqb = (int32_t)nqb;
  pp.out_bf16 = out_dtype == KVQ_DTYPE_BF16;
  pp.qk_log2 = softmax_scale * 1.4426950408889634f;
  pp.wait_ns = test_wait_limit_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)(ctas * splits);
  if (pair) return D == 128 ? launch_prefill8_d<128, true>(pp, s, grid) : launch_prefill8_d<64, true>(pp, s, grid);
  return D == 128 ? launch_prefill8_d<128, false>(pp, s, grid) : launch_prefill8_d<64, false>(pp, s, grid);
}
