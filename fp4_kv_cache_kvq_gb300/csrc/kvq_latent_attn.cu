// kvq_latent_attn.cu -- attention over the latent cache (absorbed form), one
// token per sequence or a chunk of them, on the 5th-generation tensor cores
// (tcgen05, accumulators in TMEM), and its C entry points.
//
// Mathematics.  With a token's codes and its scale s = 2^e,
//   S = q . codes,  y = S s (softmax_scale log2 e),  x = 2^(y + e - ref),
//   out = 2^-o sum x code / l,  l = sum x 2^(-e - o).
// The values' scale is a power of two and stands in x's exponent beside the
// softmax's own, so the codes enter both products as the cache holds them: a tile
// is copied once and read twice, as K-major operand (tokens x channels) for S and
// as MN-major operand (channels x tokens) for the sums.  ref, of a row's own, goes by the
// largest y + e so far, and o, if scales lie far apart, by the largest y: the same y + e,
// rounded once, and exact differences of it stand in x and in l, so that neither tiny nor
// huge values beside others, nor scores of any size, make the two differ.
//   q   scaled per row by a power of two to [2^7, 2^8), is the sum of two E4M3
//       values hi = RNE(q), lo = RNE(q - hi): exact down to 2^-9 of the row's
//       largest element, off by at most 2^-17 of it below.  hi and lo are rows of
//       one operand (128 rows for 64 queries); their scores are added in fp32.
//   x   reaches 2^3 .. 2^11 in every row and is rounded to f16, then held as a sum of
//       an E4M3 and an E5M2 value: first the rounding to E4M3 (to E5M2 over 448, E4M3's
//       end), then of the rest to the other: off by 2^-8 of x either way, or 2^-14
//       under 2^-6, where E4M3's steps end and E5M2's range (down to 2^-17) takes
//       over.  Two products of 8-bit operands cost what one of 16-bit ones costs
//       and need no expansion of the values.
// Sums, maxima and accumulators are fp32.
//
// Work.  A row is a query head of a token; a unit is 64 rows of one sequence and
// all its positions.  A CTA holds 64 rows: sum^T is 4 accumulators of 128
// channels x 64 rows (256 TMEM columns at latent_dim 512), q's latent part 128 columns,
// S two times 64; q's position part lies in shared memory.
// Few units: the positions of all sequences, laid end to end, are split evenly over
// the CTAs, the row tiles of a sequence side by side so that they read the same
// tile at the same time, and a second launch joins the parts.  Many: a unit per CTA,
// the longest first.
// Twenty warps: softmax (two groups of 8 that take every second tile; thread = two rows x
// 8 positions), loader, two that issue the products, scales, joined by mbarriers (every
// wait bounded); of a tile's steps only the choice of the references waits for the tile
// before:
//   loader    bulk copies of 64-token tiles into a ring
//   products  S(j) = q K(j)^T         kind::f8f6f4, q's latent part from TMEM; two buffers
//             O^T += K(j)^T x(j)      kind::f8f6f4, twice (hi, lo), from another warp:
//             one's waits do not hold up the other's products
//   scales    2^e, e and 2^-e of a tile's tokens, once for all rows
//
// What bounds it: for 64 rows a tile's products take 1152 cycles of the tensor pipe at its
// rate, and 1660 as they come: 39 an MMA of the scores (64 columns: the queries' rows are
// read for half the work), 53 one of the sums (A from shared memory, 4 KB each); its
// codes, 41 KB, take 1750 from HBM when every SM reads its own.  A tile takes 1900.  In
// copies with arithmetic left out the chunk took, of 1.85 ms, 1.81 without the
// conversions to 8 bits, 1.83 without the exponentials or the stores: the products, and
// the hand-offs between the groups, are what is left.  The batch of 16 heads stays where
// it is in each of these: a third of its time is start, change of unit, end and join.
// Measured (TFLOP/s of the absorbed form, 2 (2 L + R) per pair; L 512, R 64, page 64, L2
// flushed): chunk of 1024 over 8192, 2 sequences, 64 heads 1.77 ms, 1237; 64 x 8192
// positions, 16 heads 89 us, 3.8 TB/s; 16 x 32768, 128 heads 150 us, 974.
// From 3.71 ms for the chunk: softmax on eight warps instead of four 3.45; a tile's
// scales prepared by a warp of their own 3.31; MMAs issued by an elected lane 2.53;
// scores and sums issued by a warp each 2.46; the references' slack 3 -> 6 (E5M2 first
// over 448) 2.36; two groups of eight, with waits suspended in the barrier instead of
// polling, 2.07; a wait that is over looked at once 2.03; references set ahead 1.85;
// a row's references settled by its own two warps, O rescaled after the weights 1.81;
// l's form decided by the scales' warp, kTop within the references 1.77.
// Slower: A kept in the collector for the second MMA of a pair (the second one's B is then
// read in the first one's type); waits by one lane of a warp (2.79) or by one warp of a group
// (2.26); polling 64 times before suspending (3.94); four warps a group 2.35; warps
// without rows skipped (2.08: the spills cost more).
#include "kvq_latent.cuh"
#include "kvq_roles.cuh"
#include "kvq_tc.cuh"

#include <cuda_bf16.h>

namespace kvq {
namespace {

constexpr int kLT = 64;     // positions per tile
constexpr int kLRows = 64;  // query rows per unit
// softmax warps: two groups that take every second tile, two parts of a tile's positions each
constexpr int kParts = 4, kPCols = 32, kPairs = kPCols / 8, kGroupThreads = 256;
constexpr int kLSmWarps = 4 * kParts, kLSoftmax = 32 * kLSmWarps, kLThreads = kLSoftmax + 128;
constexpr int kLdWarpL = kLSmWarps, kSWarpL = kLdWarpL + 1, kOWarpL = kSWarpL + 1;  // and the scales' warp
constexpr int kPBytes = kLRows * kLT;  // one part (hi or lo) of x, one byte an element
constexpr int kMinTiles = 2;           // least tiles of a split range
// x of a row's largest product is 2^(kTop - kAhead) .. 2^(kTop + kSlackL): over 2^11.8 the rest
// behind E5M2 would leave E4M3.  (The references lie kTop under the scores: added apart it would
// be lost beside large ones.)  They are raised only past the slack, since
// that rescales O (a slack of 3: among 64 rows some raised its own in every second
// tile, 1100 cycles each).
constexpr float kTop = 5.0f, kSlackL = 6.0f;
// Where both halves of the tile that raises a reference hold products within 2^kNearL of
// each other, it is set 2^kAhead higher: larger ones will follow (chunk 2.03 -> 1.85 ms).  A
// single large one in one half is more likely the largest of all, and leaves the small
// ones beside it their distance to the end of E5M2.
constexpr float kNearL = 4.0f, kAhead = 2.0f;
constexpr float kE4m3End = 8.80f;  // a little under log2 448

enum : int {
  kLFull = 0,               // [stages] codes and exponents landed
  kLEmpty = kLFull + 8,     // [stages] the tile's sums done (commit)
  kLSFull = kLEmpty + 8,    // [stages] S in TMEM (commit), and the tile's scales ready
  kLSFree = kLSFull + 8,    // [2] S taken by the group's warps
  kLRef = kLSFree + 2,      // [2][4] the references of a quarter's rows that hold from a tile on
  kLQFull = kLRef + 8,      // q in TMEM and shared memory
  kLPFull = kLQFull + 1,    // [2] x in shared memory, O rescaled
  kLPvDone = kLPFull + 2,   // [2] O += done
  kLDrain = kLPvDone + 2,   // the last commits of the two issuing warps
  kLBars = kLDrain + 1
};

struct LatentAttnParams {
  kvq_latent_cache c;
  const int32_t* lens;
  const int32_t* chunk_lens;
  const uint16_t* q;
  void* out;
  float* part_o;    // [ctas][2][64][L]: a part's own result
  float* part_lse;  // [ctas][2][64]: log2 of its sum of weights
  int2* rec;        // [batch * tpb]: first CTA and number of parts of a unit
  int32_t* flag;
  int32_t batch, hq, chunk, out_bf16;
  int32_t tpb;      // row tiles per sequence
  int32_t groups;   // CTAs per row tile that share the positions; 0: a unit per CTA
  float scale_log2;
  uint64_t wait_ns; // a test's limit of the waits, or 0
};

template <int L, int R>
struct LGeo {
  static constexpr int kRow = L + 2 * R;
  static constexpr int kTile = kLT * kRow;
  static constexpr int kMost = (220 * 1024 - 4 * kPBytes - 128 * R) / (kTile + kLT * 13);
  static constexpr int kStages = kMost < 6 ? kMost : 6;
  static constexpr int kP = kStages * kTile;              // [2][first, second part]
  static constexpr int kQr = kP + 4 * kPBytes;            // q's position part [R / 16][16 row groups][8][16]
  static constexpr int kExp = kQr + 128 * R;              // [stages][64]
  static constexpr int kMask = kExp + kStages * kLT;      // [stages] valid tokens, 64 bits
  static constexpr int kRefS = kMask + 8 * 8;             // [64] the rows' references
  static constexpr int kAlpha = kRefS + 4 * kLRows;       // [2][2][64] factors of O's columns, by group and tile; the result's two
  static constexpr int kShare = kAlpha + 4 * 4 * kLRows;  // [2][kParts][64] what the parts of a row exchange
  static constexpr int kSc = kShare + 2 * kParts * 4 * kLRows;  // [stages][3][64] 2^e, e (-inf: no token), 2^-e
  static constexpr int kOff = kSc + kStages * 3 * 4 * kLT;  // [threads][2] l's own references
  static constexpr int kNear = kOff + 8 * kLSoftmax;  // [stages] all scales within 2^-40 .. 2^40, up to this tile
  static constexpr int kBar = kNear + 4 * 8;
  static constexpr int kMisc = kBar + 8 * kLBars;         // TMEM slot, abort, the groups' [2][2]
  static constexpr int kUsed = kMisc + 32 + 128;
  static constexpr int kBytes = kUsed > 116 * 1024 ? kUsed : 116 * 1024;  // one CTA per SM: it holds all of TMEM
  static constexpr int kOCol = 0, kQCol = L / 2, kSCol = kQCol + L / 4;
  static_assert(kSCol + 2 * kLT <= 512 && kStages >= 4 && kUsed <= 227 * 1024 && kBar % 8 == 0 && kStages <= 8, "layout");
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// Instruction descriptors: fp32 accumulators, M = 128, A E4M3, B E4M3 or E5M2.
constexpr uint32_t kIdS = (1u << 4) | (kLT / 8 << 17) | (128u / 16 << 24);
constexpr uint32_t kIdO = (1u << 4) | (1u << 15) | (128u / 16 << 24);  // A MN-major; the columns: those with rows
constexpr uint32_t kIdE5m2 = 1u << 10;                                 // B E5M2

// 16 lanes x 32 columns of TMEM, without the wait: register 4j + 2i + e holds row
// lane/4 + 8i, column 8j + 2(lane%4) + e.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// Wait for the thread's TMEM loads; a and b pass through, so their uses stay behind it.
__device__ __forceinline__ void tmem_wait_ld2(uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
               :
               : "memory");
  asm volatile(""
               : "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_16x256b_x1(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_of_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e5m2x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;\n" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t lds_f32x2(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];\n" : "=l"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts_u32x2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};\n" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void sts_f32x2(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};\n" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ __half2 u32_half2(uint32_t v) {
  __half2 h;
  *reinterpret_cast<uint32_t*>(&h) = v;
  return h;
}
__device__ __forceinline__ void sts_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
// Named barrier `id` of `threads` softmax threads; true when any thread's v is.
__device__ __forceinline__ bool softmax_or(uint32_t id, uint32_t threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ int64_t capacity(const kvq_latent_cache& c) { return (int64_t)c.max_pages_per_seq * c.page_size; }

// Tiles that sequence b takes on the line of all sequences' positions (1 at least).
__device__ __forceinline__ int64_t line_tiles(const LatentAttnParams& p, int b) {
  const int64_t t = min((int64_t)max(__ldg(p.lens + b), 0), capacity(p.c));
  return max((int64_t)1, (t + kLT - 1) / kLT);
}

// One CTA's share of a unit: tiles [t0, t1) of the nt that its rows attend.
struct Unit {
  int b, r, rows, n, t0, t1;
  int64_t first, limit;  // position of the chunk's token 0; positions read
  bool whole;
  int slot;
};

// The CTA's range of the line of all sequences' tiles: sequence b starts at `base` of it.
struct Plan {
  int64_t lo, hi, base, per;
  int b;
};

// Every warp finds it for itself, so that none waits for another's.
__device__ __forceinline__ Plan find_plan(const LatentAttnParams& p, int lane) {
  Plan r = {0, 0, 0, 1, 0};
  if (p.groups == 0) return r;
  int64_t total = 0;
  for (int b = lane; b - lane < p.batch; b += 32)
    total += __reduce_add_sync(0xFFFFFFFFu, b < p.batch ? (uint32_t)line_tiles(p, b) : 0u);  // 2^25 each at most
  const int64_t up = total + p.groups - 1;
  r.per = max((int64_t)kMinTiles, up >> 32 ? up / p.groups : (int64_t)((uint32_t)up / (uint32_t)p.groups));
  r.lo = (int64_t)(blockIdx.x / (unsigned)p.tpb) * r.per;
  if (r.lo >= total) return r;
  r.hi = min(r.lo + r.per, total);
  for (int b = lane; b - lane < p.batch; b += 32) {
    const uint32_t c = b < p.batch ? (uint32_t)line_tiles(p, b) : 0u;
    uint32_t pre = c;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, pre, o);
      if (lane >= o) pre += x;
    }
    const uint32_t sum = __shfl_sync(0xFFFFFFFFu, pre, 31);
    if (r.lo < r.base + sum) {
      const int at = __ffs(__ballot_sync(0xFFFFFFFFu, r.lo < r.base + pre)) - 1;
      r.base += __shfl_sync(0xFFFFFFFFu, pre - c, at);
      r.b = b - lane + at;
      break;
    }
    r.base += sum;
  }
  return r;
}

// The CTA's units in order; every role walks them alike.
struct Walk {
  const LatentAttnParams& p;
  int64_t lo, hi, base, per, i;
  int b;
  __device__ Walk(const LatentAttnParams& p_, const Plan& pl)
      : p(p_), lo(pl.lo), hi(pl.hi), base(pl.base), per(pl.per), i(blockIdx.x), b(pl.b) {}
  __device__ void rows_of(Unit& u, int32_t* flag) const {
    const int32_t T = __ldg(p.lens + u.b), n = p.chunk_lens ? __ldg(p.chunk_lens + u.b) : p.chunk;
    const bool decode = p.chunk == 1 && p.chunk_lens == nullptr;
    const bool bad_n = n < 0 || n > p.chunk;
    if ((bad_n || T < (decode ? 0 : n)) && u.r == 0) set_flag(flag, KVQ_FLAG_BAD_LENGTH);
    u.n = bad_n ? 0 : n;
    u.rows = (int)max((int64_t)0, min((int64_t)kLRows, (int64_t)u.n * p.hq - (int64_t)u.r * kLRows));
    u.first = (int64_t)T - u.n;
    u.limit = 0;
    if (u.rows > 0 && u.first >= 0) {
      u.limit = u.first + (u.r * kLRows + u.rows - 1) / p.hq + 1;
      if (u.limit > capacity(p.c)) {
        u.limit = capacity(p.c);
        set_flag(flag, KVQ_FLAG_PAGE_OOB);
      }
    }
  }
  // flag: where bad lengths are reported (one role does)
  __device__ bool next(Unit& u, int32_t* flag) {
    while (true) {
      if (p.groups == 0) {
        if (i >= (int64_t)p.batch * p.tpb) return false;
        u.r = p.tpb - 1 - (int)(i / p.batch);
        u.b = (int)(i % p.batch);
        i += gridDim.x;
        rows_of(u, flag);
        u.t0 = 0;
        u.t1 = (int)((u.limit + kLT - 1) / kLT);
        u.whole = true;
        u.slot = 0;
      } else {
        if (base >= hi) return false;
        const int64_t cost = line_tiles(p, b);
        const int64_t s0 = max(lo - base, (int64_t)0), s1 = min(hi - base, cost);
        u.b = b;
        u.r = (int)(blockIdx.x % (unsigned)p.tpb);
        rows_of(u, flag);
        const int nt = (int)((u.limit + kLT - 1) / kLT);
        u.t0 = (int)min(s0, (int64_t)nt);
        u.t1 = (int)min(s1, (int64_t)nt);
        u.whole = s0 == 0 && s1 == cost;
        u.slot = s0 > 0 ? 0 : 1;
        if (flag == p.flag && s0 == 0 && threadIdx.x == 0) {
          const int64_t span = base - lo + cost - 1;  // ranges that it reaches beyond this one: span / per
          const int more = span < per ? 0 : span >> 32 ? (int)(span / per) : (int)((uint32_t)span / (uint32_t)per);
          p.rec[(int64_t)b * p.tpb + u.r] = make_int2((int)blockIdx.x, more + 1);
        }
        base += cost;
        ++b;
      }
      if (u.rows > 0) return true;
    }
  }
};

template <int L, int R>
__global__ void __launch_bounds__(kLThreads, 1) latent_attn_kernel(const LatentAttnParams p) {
  using G = LGeo<L, R>;
  constexpr int kM = L / 128, kSteps = (L + R) / 32;
  extern __shared__ uint8_t lat_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lat_raw) + 127) & ~uintptr_t(127));
  const uint32_t sb = smem_addr(base), bars = sb + G::kBar;
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + G::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* near_s = reinterpret_cast<volatile int*>(base + G::kNear);
  volatile uint64_t* vmask = reinterpret_cast<volatile uint64_t*>(base + G::kMask);
  const BoundedWaits wait{abort, p.wait_ns};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(bars + 8 * (kLFull + s), 1);
      mbar_init(bars + 8 * (kLEmpty + s), 1);
      mbar_init(bars + 8 * (kLSFull + s), 2);
    }
    mbar_init(bars + 8 * kLQFull, kLSmWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (kLSFree + i), kLSmWarps / 2);
      for (int k = 0; k < 4; ++k) mbar_init(bars + 8 * (kLRef + 4 * i + k), 2);
      mbar_init(bars + 8 * (kLPFull + i), kLSmWarps / 2);
      mbar_init(bars + 8 * (kLPvDone + i), 1);
    }
    mbar_init(bars + 8 * kLDrain, 2);
    *abort = 0;
    misc[2] = misc[3] = misc[4] = misc[5] = 0u;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(smem_addr(misc), 512);
  Walk walk(p, find_plan(p, lane));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);
  Unit u;
  bool failed = false;

  if (warp < kLSmWarps) {
    // ------------------------------------------------------------ softmax
    // warp w: rows 16 (w & 3) .. + 15, whose scores lie in its 32 TMEM lanes; of every
    // second tile (w >> 3) the positions 32 (w >> 2 & 1) .. + 31
    const int g = lane >> 2, t = lane & 3, quad = warp & 3, share = warp >> 2, part = share & 1;
    const uint32_t grp = (uint32_t)share >> 1, bar_g = 2 + grp, bar_r = 4 + 4 * grp + quad;  // named barriers: the group's, a row's two warps'
    const uint32_t tw = tmem + ((uint32_t)(32 * quad) << 16);
    const int lr[2] = {16 * quad + g, 16 * quad + g + 8};
    float* ref_s = reinterpret_cast<float*>(base + G::kRefS);
    float* alpha = reinterpret_cast<float*>(base + G::kAlpha);
    float* shared = reinterpret_cast<float*>(base + G::kShare);  // [2][kParts][64]
    float* own = shared + share * kLRows;
    volatile int* gave_up = reinterpret_cast<volatile int*>(misc) + 2 + 2 * grp;  // [2] a wait of the group did, by its tile's parity
    const uint32_t off = sb + G::kOff + 8 * tid;
    uint32_t it0 = 0;  // tiles before the unit
    while (walk.next(u, tid == 0 ? p.flag : nullptr)) {
      const int64_t row0 = (int64_t)u.b * p.chunk * p.hq + (int64_t)u.r * kLRows;
      if (u.t0 >= u.t1) {  // nothing attended: zero rows, or a part without weight
        if (u.whole) {
          for (int i = tid; i < u.rows * (L / 4); i += kLSoftmax) {
            const int64_t at = row0 * L + 4 * (int64_t)i;
            if (p.out_bf16)
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(0u, 0u);
            else
              *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        } else if (tid < kLRows) {
          p.part_lse[((int64_t)blockIdx.x * 2 + u.slot) * kLRows + tid] = -INFINITY;
        }
        continue;
      }
      // q: four lanes share a row's 64-byte pieces, a part takes every fourth one; hi to lanes 0..15, lo to lanes 16..31 of the quarter's TMEM lanes
      constexpr int kOwn = (kSteps + kParts - 1) / kParts;
      uint4 qv[2][kOwn];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          const int s = kParts * k + share;
          qv[i][k] = make_uint4(0u, 0u, 0u, 0u);
          if (lr[i] < u.rows && s < kSteps)
            qv[i][k] = __ldg(reinterpret_cast<const uint4*>(p.q + (row0 + lr[i]) * (L + R) + 32 * s + 8 * t));
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t am = 0u;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          const uint32_t w[4] = {qv[i][k].x, qv[i][k].y, qv[i][k].z, qv[i][k].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) am = max(am, max(w[c] << 16 & 0x7FFFFFFFu, w[c] & 0x7FFF0000u));
        }
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        if (t == 0) own[lr[i]] = __uint_as_float(am);
      }
      if (tid < kLRows) ref_s[tid] = -INFINITY;
      named_barrier_sync(1, kLSoftmax);
      float xs[2];      // S to log2 units, before the token's scale
      int64_t last[2];  // last position that the row attends
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* ams = shared + lr[i];
        const uint32_t am = max(max(__float_as_uint(ams[0]), __float_as_uint(ams[kLRows])),
                                max(__float_as_uint(ams[2 * kLRows]), __float_as_uint(ams[3 * kLRows])));
        const int ex = min(max((int)(am >> 23), 8), 254);  // times 2^(134 - ex): to [2^7, 2^8)
        const bool bad = am >= 0x7F800000u;  // an Inf or NaN: the row's scores are NaN, its codes 0
        const float mul = __uint_as_float((uint32_t)(261 - ex) << 23);
        xs[i] = bad ? __uint_as_float(0x7FFFFFFFu) : p.scale_log2 * __uint_as_float((uint32_t)(ex - 7) << 23);
        last[i] = lr[i] < u.rows ? u.first + (u.r * kLRows + lr[i]) / p.hq : -1;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {  // in place: x, y the hi codes, z, w the lo codes
          if (bad) qv[i][k] = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {qv[i][k].x, qv[i][k].y, qv[i][k].z, qv[i][k].w};
          uint32_t h[4], l[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float x0 = bf16_lo(w[c]) * mul, x1 = bf16_hi(w[c]) * mul;
            h[c] = e4m3x2_from_f32(x0, x1);
            const float2 y = f16x2_to_float2(f16x2_from_e4m3x2(h[c]));
            l[c] = e4m3x2_from_f32(x0 - y.x, x1 - y.y);
          }
          qv[i][k] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, l[0] | l[1] << 16, l[2] | l[3] << 16);
        }
      }
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const int s = kParts * k + share;
        if (s < L / 32) {
          tmem_st_16x256b_x1(tw + G::kQCol + 8 * s, qv[0][k].x, qv[0][k].y, qv[1][k].x, qv[1][k].y);
          tmem_st_16x256b_x1(tw + (16u << 16) + G::kQCol + 8 * s, qv[0][k].z, qv[0][k].w, qv[1][k].z, qv[1][k].w);
        } else if (s < kSteps) {  // the position part: row 32 quad + 16 (lo) + its number, as the TMEM lanes
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = sb + G::kQr + (uint32_t)((2 * (s - L / 32) + (t >> 1)) * 2048 + (4 * quad + i) * 128 +
                                                         g * 16 + (t & 1) * 8);
            sts_u32x2(at, qv[i][k].x, qv[i][k].y);
            sts_u32x2(at + 256, qv[i][k].z, qv[i][k].w);
          }
        }
      }
      fence_async_smem();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * kLQFull);

      // l counts x 2^(-e - o) over the reference m of the thread's last tile.  Short form: o
      // is 0.  That would lose what scales far apart leave under fp32's range: from the unit's
      // first tile with a scale outside 2^-40 .. 2^40 on, o goes by the thread's own largest
      // (y + e - m) - e, with exponentials of its own; in both groups, whichever has that
      // tile, since it raises the references that they share, and over such a one a sum in
      // the short form would become 0.
      float m[2] = {-INFINITY, -INFINITY};
      sts_f32x2(off, 0.0f, 0.0f);
      uint64_t l2[2] = {0ull, 0ull};
      const int64_t full_upto = min(u.limit, u.first + (u.r * kLRows) / p.hq + 1);  // attended by every row
      bool ready = false;  // the group's next tile's scores are there
      for (int j = u.t0 + (int)((grp ^ it0) & 1u); j < u.t1; j += 2) {
        const uint32_t it = it0 + (uint32_t)(j - u.t0);
        const int st = (int)(it % G::kStages);
        if (!ready && !failed) failed = !wait(bars + 8 * (kLSFull + st), (it / G::kStages) & 1u);
        tc_fence_after();
        uint32_t v[16], lo[16];
        tmem_ld_16x256b_x4(tw + G::kSCol + kLT * grp + kPCols * part, v);
        tmem_ld_16x256b_x4(tw + (16u << 16) + G::kSCol + kLT * grp + kPCols * part, lo);
        const bool near = near_s[st] != 0;  // (the long form up to the unit's end)
        const uint32_t sc = sb + G::kSc + (uint32_t)(st * 3 * 4 * kLT + 4 * (kPCols * part + 2 * t));
        uint64_t s2[kPairs], x2[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          s2[k] = lds_f32x2(sc + 32 * k);
          x2[k] = lds_f32x2(sc + 4 * kLT + 32 * k);
        }
        const int64_t p0 = (int64_t)j * kLT;
        const bool partly = p0 + kLT > full_upto;  // some row sees the tile in part
        tmem_wait_ld2(v, lo);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (kLSFree + grp));
        uint64_t z2[2][kPairs];
        float top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            const uint64_t S = add2(pack2(__uint_as_float(v[4 * k + 2 * i]), __uint_as_float(v[4 * k + 2 * i + 1])),
                                    pack2(__uint_as_float(lo[4 * k + 2 * i]), __uint_as_float(lo[4 * k + 2 * i + 1])));
            z2[i][k] = fma2(S, mul2(pack2(xs[i], xs[i]), s2[k]), x2[k]);
          }
          if (partly) {
            const int lim = (int)max((int64_t)-1, min((int64_t)kLT, last[i] - p0)) - kPCols * part - 2 * t;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
              const float2 f = unpack2(z2[i][k]);
              z2[i][k] = pack2(8 * k > lim ? -INFINITY : f.x, 8 * k + 1 > lim ? -INFINITY : f.y);
            }
          }
          const float2 a = unpack2(z2[i][0]), b = unpack2(z2[i][1]), c = unpack2(z2[i][2]), d = unpack2(z2[i][3]);
          top[i] = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)), fmaxf(fmaxf(c.x, c.y), fmaxf(d.x, d.y)));
        }
        // (waits that are over are known to be by the time they are due: a look takes 150 cycles)
        const bool x_free = it < 2 || wait.over(bars + 8 * (kLPvDone + grp), ((it >> 1) - 1) & 1u);
        if (j > u.t0 && !failed) failed = !wait(bars + 8 * (kLRef + 4 * (grp ^ 1) + quad), ((it - 1) >> 1) & 1u);
        float ref[2];
        bool up = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ref[i] = ref_s[lr[i]];
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
          up |= top[i] - ref[i] > kTop + kSlackL;
        }
        // raise the references of the rows that need it (what a row gives does not depend on
        // others); a row's two warps agree, the other group's wait for them
        float* fac = alpha + (2 * grp + (it >> 1 & 1)) * kLRows;
        float a2[2] = {1.0f, 1.0f};
        const bool raised = softmax_or(bar_r, 64, up);
        if (raised) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (t == 0) own[kParts * kLRows + lr[i]] = top[i];
          named_barrier_sync(bar_r, 64);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float* x = shared + (kParts + 2 * grp) * kLRows + lr[i];
            const float all = fmaxf(x[0], x[kLRows]), other = fminf(x[0], x[kLRows]);
            const float ahead = other > all - kNearL ? kAhead : 0.0f;
            const float to = all - ref[i] > kTop + kSlackL ? floorf(all) + (ahead - kTop) : ref[i];
            a2[i] = to == ref[i] ? 1.0f : fast_exp2(ref[i] - to);
            if (t == 0 && part == 0) ref_s[lr[i]] = to;
            ref[i] = to;
          }
        }
        if (t == 0 && part == 0) fac[lr[0]] = a2[0], fac[lr[1]] = a2[1];
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (kLRef + 4 * grp + quad));
        // x in two parts to shared memory, [16 tokens][8 rows] core matrices, once the sums
        // of the tile before last have read theirs
        if (!__all_sync(0xFFFFFFFFu, x_free) && !failed)
          failed = !wait(bars + 8 * (kLPvDone + grp), ((it >> 1) - 1) & 1u);
        const uint32_t nx = it + 2;  // a look at the next wait, ahead of its time: it takes 150 cycles
        ready = j + 2 < u.t1 && wait.over(bars + 8 * (kLSFull + nx % G::kStages), (nx / G::kStages) & 1u);
        // (all of a thread's loads, then its arithmetic, then its stores: they keep their order, and
        // one pair after the other would wait for each one's chain of conversions)
        uint64_t inv2[kPairs];
        uint32_t w[2][kPairs];  // first part | second part << 16
#pragma unroll
        for (int k = 0; k < kPairs; ++k) inv2[k] = lds_f32x2(sc + 8 * kLT + 32 * k);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float rf = ref[i] == -INFINITY ? 0.0f : -ref[i];
          const bool large = __any_sync(0xFFFFFFFFu, top[i] + rf > kE4m3End);  // some x is over 448: E5M2 first
          const float raise = m[i] == ref[i] ? 0.0f : m[i] - ref[i];  // since the group's last tile
          m[i] = ref[i];
#pragma unroll
          for (int k = 0; k < kPairs; ++k) z2[i][k] = add2(z2[i][k], pack2(rf, rf));
          if (near) {
            const float a = fast_exp2(raise);
            l2[i] = mul2(l2[i], pack2(a, a));
          } else {
            const float o = lds_f32(off + 4 * i) + raise;
            float to = o;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
              const float2 f = unpack2(z2[i][k]), x = unpack2(x2[k]);
              to = fmaxf(to, fmaxf(x.x == -INFINITY ? x.x : f.x - x.x, x.y == -INFINITY ? x.y : f.y - x.y));
            }
            const float zero = to == -INFINITY ? 0.0f : to, a = fast_exp2(o - zero);
            l2[i] = mul2(l2[i], pack2(a, a));
            sts_f32(off + 4 * i, to);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
              const float2 f = unpack2(z2[i][k]), x = unpack2(x2[k]);
              l2[i] = add2(l2[i], pack2(x.x == -INFINITY ? 0.0f : fast_exp2((f.x - x.x) - zero),
                                        x.y == -INFINITY ? 0.0f : fast_exp2((f.y - x.y) - zero)));
            }
          }
          uint64_t sum = 0ull;
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            const float2 f = unpack2(z2[i][k]);
            const float xa = fast_exp2(f.x), xb = fast_exp2(f.y);
            sum = fma2(pack2(xa, xb), inv2[k], sum);
            const uint32_t h = pack_f16x2(xa, xb);
            uint32_t hi = e4m3x2_of_f16x2(h);
            uint32_t rest = e5m2x2_of_f16x2(hsub2(h, f16x2_from_e4m3x2(hi)));
            if (large) {
              const uint32_t r = e5m2x2_of_f16x2(h), q = e4m3x2_of_f16x2(hsub2(h, f16x2_of_e5m2x2(r)));
              const uint32_t over = prmt(__hgt2_mask(u32_half2(h), u32_half2(0x5F005F00u)), 0u, 0x4420u);  // 448
              hi = (hi & ~over) | (q & over);
              rest = (rest & ~over) | (r & over);
            }
            w[i][k] = hi | rest << 16;
          }
          if (near) l2[i] = add2(sum, l2[i]);
        }
        const uint32_t pb = sb + G::kP + (it & 1) * 2 * kPBytes + (uint32_t)(part * 2048 + 2 * t);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            const uint32_t a = pb + (uint32_t)((lr[i] >> 3) * 128 + (lr[i] & 7) * 16 + (k >> 1) * 1024 + (k & 1) * 8);
            sts_u16(a, w[i][k]);
            sts_u16(a + kPBytes, w[i][k] >> 16);
          }
        ready = __all_sync(0xFFFFFFFFu, ready);
        fence_async_smem();
        // O's columns follow (none at the unit's first tile): all warps, since each holds a
        // quarter of the channels
        if (failed) gave_up[it >> 1 & 1] = 1;
        if (softmax_or(bar_g, kGroupThreads, raised || failed)) {
          if (gave_up[it >> 1 & 1]) {
            failed = true;
            break;
          }
          if (j > u.t0) {
            failed = !wait(bars + 8 * (kLPvDone + (grp ^ 1)), ((it - 1) >> 1) & 1u);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 2 * kM; ++c) {
              uint32_t o[16];
              const int col = 32 * part + 16 * (c & 1);
              const uint32_t at = tw + G::kOCol + kLRows * (c >> 1) + col;
              tmem_ld16(at, o);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float4 a = *reinterpret_cast<const float4*>(fac + col + 4 * k);
                o[4 * k] = __float_as_uint(__uint_as_float(o[4 * k]) * a.x);
                o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * a.y);
                o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * a.z);
                o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * a.w);
              }
              tmem_st16_async(at, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        __syncwarp();
        if (lane == 0 && !failed) mbar_arrive(bars + 8 * (kLPFull + grp));
      }
      // the unit's result: O / l, l over the row's parts and for one offset of all from the
      // row's last reference
      it0 += (uint32_t)(u.t1 - u.t0);
      if (!failed) failed = !wait(bars + 8 * (kLPvDone + ((it0 - 1) & 1)), ((it0 - 1) >> 1) & 1u);
      if (softmax_or(1, kLSoftmax, failed)) {
        failed = true;  // (in every softmax warp)
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float r = ref_s[lr[i]];
        m[i] = lds_f32(off + 4 * i) + (m[i] == r ? 0.0f : m[i] - r);
        float mq = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], 1));
        mq = fmaxf(mq, __shfl_xor_sync(0xFFFFFFFFu, mq, 2));
        if (t == 0) own[kParts * kLRows + lr[i]] = mq;
      }
      named_barrier_sync(1, kLSoftmax);
      float mm[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* ms = shared + kParts * kLRows + lr[i];
        const float all = fmaxf(fmaxf(ms[0], ms[kLRows]), fmaxf(ms[2 * kLRows], ms[3 * kLRows]));
        mm[i] = all == -INFINITY ? 0.0f : all;
        const float2 x = unpack2(l2[i]);
        float l = (x.x + x.y) * fast_exp2(m[i] - mm[i]);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if (t == 0) own[lr[i]] = l;
      }
      named_barrier_sync(1, kLSoftmax);
      if (t == 0 && share == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* x = shared + lr[i];
          const float r = ref_s[lr[i]];
          const float l = (x[0] + x[kLRows]) + (x[2 * kLRows] + x[3 * kLRows]);
          const float d = -mm[i], h = rintf(0.5f * d);
          alpha[lr[i]] = fast_exp2(h);  // two factors: 2^d alone can leave fp32's range
          alpha[kLRows + lr[i]] = l == 0.0f ? 0.0f : fast_exp2(d - h) / l;
          if (!u.whole)
            p.part_lse[((int64_t)blockIdx.x * 2 + u.slot) * kLRows + lr[i]] = l == 0.0f ? -INFINITY : (r == -INFINITY ? 0.0f : r) + (mm[i] + log2f(l));
        }
      }
      named_barrier_sync(1, kLSoftmax);
      float* po = p.part_o + ((int64_t)blockIdx.x * 2 + u.slot) * kLRows * L;
      // (128 channels of 16 rows at a time, the warps of a quarter in turn)
#pragma unroll 1
      for (int c = share; c < 4 * kM; c += kParts) {
        const int mm = c % kM, c0 = 16 * (c / kM), there = u.rows - c0, ch = 128 * mm + 32 * quad + lane;
        if (there <= 0) break;
        uint32_t o[16];
        float4 fa[4], fb[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          fa[k] = *reinterpret_cast<const float4*>(alpha + c0 + 4 * k);
          fb[k] = *reinterpret_cast<const float4*>(alpha + kLRows + c0 + 4 * k);
        }
        tmem_ld16(tw + G::kOCol + kLRows * mm + c0, o);
        const auto scaled = [&](int k, float a, float b) { return b == 0.0f ? 0.0f : __uint_as_float(o[k]) * a * b; };
        float x[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[4 * k] = scaled(4 * k, fa[k].x, fb[k].x), x[4 * k + 1] = scaled(4 * k + 1, fa[k].y, fb[k].y);
          x[4 * k + 2] = scaled(4 * k + 2, fa[k].z, fb[k].z), x[4 * k + 3] = scaled(4 * k + 3, fa[k].w, fb[k].w);
        }
        if (!u.whole) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k < there) po[(c0 + k) * L + ch] = x[k];
        } else if (p.out_bf16) {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (row0 + c0) * L + ch;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k < there) out[k * L] = __float2bfloat16_rn(x[k]);
        } else {
          float* out = static_cast<float*>(p.out) + (row0 + c0) * L + ch;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k < there) out[k * L] = x[k];
        }
      }
      tc_fence_before();
      named_barrier_sync(1, kLSoftmax);  // alpha and what the halves exchanged are free again
    }
    // after a wait that gave up the walk ends without work: the join reads the record of each
    // unit, which next() writes, and each part's sum of weights (of an empty one no result)
    if (failed) {
      do {
        if (!u.whole && tid < kLRows) p.part_lse[((int64_t)blockIdx.x * 2 + u.slot) * kLRows + tid] = -INFINITY;
      } while (walk.next(u, tid == 0 ? p.flag : nullptr));
    }
  } else if (warp == kLdWarpL) {
    // ------------------------------------------------------------ loader
    const LatentLayout lay(p.c);
    const int gs = lay.G, ngs = __ffs(kLT / gs) - 1, ng = 1 << ngs, tb = 32 >> ngs;  // groups per tile, tiles per lookup
    const uint8_t* pool = static_cast<const uint8_t*>(p.c.data);
    uint32_t it = 0;
    while (!failed && walk.next(u, nullptr)) {
      int64_t off = -1;
      for (int j = u.t0; j < u.t1; ++j, ++it) {
        const int st = (int)(it % G::kStages), k = (j - u.t0) & (tb - 1);
        if (k == 0) {
          const int64_t pos = (int64_t)(j + (lane >> ngs)) * kLT + (lane & (ng - 1)) * gs;
          off = pos < u.limit && j + (lane >> ngs) < u.t1 ? latent_group(p.c, lay, u.b, pos, p.flag) : -1;
          if (off >= 0 && !KVQ_IN(off + lay.group_bytes() <= p.c.num_pages * lay.page_bytes(), p.flag)) off = -1;
        }
        const int64_t src = __shfl_sync(0xFFFFFFFFu, off, (k * ng + lane) & 31);
        const int cnt = lane < ng && src >= 0
                            ? (int)max((int64_t)0, min((int64_t)gs, u.limit - ((int64_t)j * kLT + lane * gs)))
                            : 0;
        const uint32_t code_bytes = (uint32_t)((cnt + 7) & ~7) * G::kRow;
        const uint32_t bytes = __reduce_add_sync(0xFFFFFFFFu, cnt > 0 ? code_bytes + (uint32_t)gs : 0u);
        const uint64_t bits = cnt > 0 ? (cnt >= 64 ? ~0ull : ((1ull << cnt) - 1ull) << (lane * gs)) : 0ull;
        const uint64_t ok = (uint64_t)__reduce_or_sync(0xFFFFFFFFu, (uint32_t)(bits >> 32)) << 32 |
                            __reduce_or_sync(0xFFFFFFFFu, (uint32_t)bits);
        if (it >= G::kStages && !wait(bars + 8 * (kLEmpty + st), (it / G::kStages - 1) & 1u)) {
          failed = true;
          break;
        }
        if (lane == 0) {
          vmask[st] = ok;
          mbar_arrive_expect_tx(bars + 8 * (kLFull + st), bytes);
        }
        __syncwarp();
        if (cnt > 0) {
          bulk_g2s(sb + st * G::kTile + lane * gs * G::kRow, pool + src, code_bytes, bars + 8 * (kLFull + st));
          bulk_g2s(sb + G::kExp + st * kLT + lane * gs, pool + src + lay.exponent(0), gs, bars + 8 * (kLFull + st));
        }
      }
    }
    // no copy outlives the CTA
    for (uint32_t s = it > G::kStages ? it - G::kStages : 0u; s < it; ++s) {
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait_hint(bars + 8 * (kLFull + s % G::kStages), (s / G::kStages) & 1u, 20000u) &&
             global_ns() - t0 < 20000000ull) {
      }
    }
  } else if (warp == kSWarpL || warp == kOWarpL) {
    uint32_t it = 0;
    if (warp == kSWarpL) {
      // ---------------------------------------------------------- scores
      const uint64_t dk = smem_desc(sb, 128, 8 * G::kRow);  // tokens as rows: K-major
      const uint64_t dq = smem_desc(sb + G::kQr, 2048, 128);
      uint32_t un = 0;
      while (!failed && walk.next(u, nullptr)) {
        if (u.t0 >= u.t1) continue;
        if (!wait(bars + 8 * kLQFull, un & 1u)) break;
        ++un;
        for (int j = u.t0; j < u.t1; ++j, ++it) {
          const int st = (int)(it % G::kStages);
          if (!wait(bars + 8 * (kLFull + st), (it / G::kStages) & 1u) ||
              (it > 1 && !wait(bars + 8 * (kLSFree + (it & 1)), ((it >> 1) - 1) & 1u))) {
            failed = true;
            break;
          }
          const uint64_t ok = vmask[st];
          if (ok != ~0ull) {  // rows without a token: no NaN there may reach a score or meet a weight of 0
            const uint32_t tile = sb + st * G::kTile;
            for (int i = lane; i < kLT * (G::kRow / 16); i += 32) {
              const int tok = (i & 7) | (i / (8 * (G::kRow / 16))) << 3, unit = i / 8 % (G::kRow / 16);
              if (!((ok >> tok) & 1ull))
                sts128(tile + (tok >> 3) * 8 * G::kRow + unit * 128 + (tok & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
            }
            fence_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          if (elect_one_of_warp()) {
            const uint64_t kd = dk + (uint64_t)(st * (G::kTile >> 4));
            const uint32_t d = tmem + G::kSCol + kLT * (it & 1);
#pragma unroll
            for (int s = 0; s < L / 32; ++s)
              mma_f8_ta(d, tmem + G::kQCol + 8 * s, kd + (uint64_t)(s * 256 >> 4), kIdS, s > 0);
#pragma unroll
            for (int s = 0; s < 2 * R / 32; ++s)  // the key part's hi and lo codes meet the same q
              mma_f8(d, dq + (uint64_t)(s % (R / 32) * 4096 >> 4), kd + (uint64_t)((L / 32 + s) * 256 >> 4), kIdS, true);
            tc_commit(bars + 8 * (kLSFull + st));
          }
          __syncwarp();
        }
      }
    } else {
      // ---------------------------------------------------------- sums: O^T (+)= K(j)^T x(j)
      const uint64_t dv = smem_desc(sb, 8 * G::kRow, 128);  // channels as rows: MN-major
      const uint64_t dp = smem_desc(sb + G::kP, 1024, 128);
      while (!failed && walk.next(u, nullptr)) {
        const uint32_t id = kIdO | (uint32_t)((u.rows + 15) / 16 * 2) << 17;
        for (int j = u.t0; j < u.t1; ++j, ++it) {
          if (!wait(bars + 8 * (kLPFull + (it & 1)), (it >> 1) & 1u)) {
            failed = true;
            break;
          }
          tc_fence_after();
          const int st = (int)(it % G::kStages);
          const bool more = j > u.t0;
          if (elect_one_of_warp()) {
            const uint64_t a = dv + (uint64_t)(st * (G::kTile >> 4));
            const uint64_t b = dp + (uint64_t)((it & 1) * (2 * kPBytes >> 4));
#pragma unroll
            for (int mm = 0; mm < kM; ++mm)
#pragma unroll
              for (int s = 0; s < 2; ++s) {  // 32 tokens: four core matrices of the tile, two of x
                const uint64_t am = a + (uint64_t)((mm * 1024 + s * 32 * G::kRow) >> 4);
                mma_f8(tmem + G::kOCol + mm * kLRows, am, b + (uint64_t)(s * 2048 >> 4), id, more || s > 0);
                mma_f8(tmem + G::kOCol + mm * kLRows, am, b + (uint64_t)((s * 2048 + kPBytes) >> 4), id | kIdE5m2, true);
              }
            tc_commit(bars + 8 * (kLEmpty + st));
            tc_commit(bars + 8 * (kLPvDone + (it & 1)));
          }
          __syncwarp();
        }
      }
    }
    // no product outlives the CTA (a commit covers its own thread's, so the lane that issued them makes it)
    __syncwarp();
    if (elect_one_of_warp()) tc_commit(bars + 8 * kLDrain);
    __syncwarp();
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait_hint(bars + 8 * kLDrain, 0u, 20000u) && global_ns() - t0 < 20000000ull) {
    }
  } else {
    // ------------------------------------------------------------ scales
    uint32_t it = 0;
    while (!failed && walk.next(u, nullptr)) {
      bool near = true;  // the unit's tiles so far
      for (int j = u.t0; j < u.t1; ++j, ++it) {
        const int st = (int)(it % G::kStages);
        if (!wait(bars + 8 * (kLFull + st), (it / G::kStages) & 1u)) {
          failed = true;
          break;
        }
        const uint64_t ok = vmask[st];
        const uint32_t sc = sb + G::kSc + (uint32_t)(st * 3 * 4 * kLT + 8 * lane);
        const uint32_t e2 = lds16(sb + G::kExp + st * kLT + 2 * lane);
        float s[2], x[2], inv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t e = i ? e2 >> 8 : e2 & 0xFFu;
          const bool in = (ok >> (2 * lane + i)) & 1ull;
          s[i] = in ? latent_scale(e) : 1.0f;
          x[i] = in ? (float)((int)e - 127) : -INFINITY;
          inv[i] = in ? __uint_as_float((254u - e) << 23) : 1.0f;
          near = near && (!in || e - 87u <= 80u);  // 2^-40 .. 2^40
        }
        sts_f32x2(sc, s[0], s[1]);
        sts_f32x2(sc + 4 * kLT, x[0], x[1]);
        sts_f32x2(sc + 8 * kLT, inv[0], inv[1]);
        near = __all_sync(0xFFFFFFFFu, near);
        if (lane == 0) near_s[st] = near;
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (kLSFull + st));
      }
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

// Joins the parts of units that several CTAs worked on, out = sum w_i o_i, w_i =
// 2^(lse_i - m) / sum 2^(lse_j - m): a CTA per row, its warps take every fourth part, two
// at a time, and add up in a fixed order.
template <int L>
__global__ void __launch_bounds__(128) latent_merge_kernel(const LatentAttnParams p, int rows_per_unit) {
  __shared__ float acc_s[4][L];
  __shared__ float l_s[4];
  const int unit = blockIdx.x / rows_per_unit, r = blockIdx.x % rows_per_unit, lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5, b = unit / p.tpb, rt = unit % p.tpb;
  const int n = p.chunk_lens ? __ldg(p.chunk_lens + b) : p.chunk;
  grid_dependency_wait();
  if (n < 0 || n > p.chunk || (int64_t)rt * kLRows + r >= (int64_t)n * p.hq) return;
  const int2 rec = p.rec[unit];
  // (looked at in every build: the record is in the caller's memory, and all reads go by it)
  const int ctas = p.groups * p.tpb;
  const bool inside = rec.y <= p.groups && rec.x >= 0 && rec.x < ctas && rec.x + (rec.y - 1) * p.tpb < ctas;
  if (rec.y <= 1 || !KVQ_IN(inside, p.flag) || !inside) return;
  const auto at = [&](int i) { return ((int64_t)(rec.x + i * p.tpb) * 2 + (i == 0 ? 1 : 0)) * kLRows + r; };
  float m = -INFINITY;
  for (int i = lane; i < rec.y; i += 32) m = fmaxf(m, p.part_lse[at(i)]);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float mm = m == -INFINITY ? 0.0f : m;
  float acc[L / 32], l = 0.0f;
#pragma unroll
  for (int c = 0; c < L / 32; ++c) acc[c] = 0.0f;
  for (int i = warp; i < rec.y; i += 8) {
    const int64_t a[2] = {at(i), at(i + 4 < rec.y ? i + 4 : i)};
    float4 v[2][L / 128];
    float w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      w[k] = p.part_lse[a[k]];
#pragma unroll
      for (int c = 0; c < L / 128; ++c) v[k][c] = (reinterpret_cast<const float4*>(p.part_o + a[k] * L) + lane)[32 * c];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (w[k] == -INFINITY || (k == 1 && i + 4 >= rec.y)) continue;  // (a part without weight left no result)
      const float x = fast_exp2(w[k] - mm) * (1.0f / 256.0f);  // (fewer parts than 256: sum x o stays in fp32 for any o)
      l += x;
#pragma unroll
      for (int c = 0; c < L / 128; ++c) {
        acc[4 * c] += x * v[k][c].x, acc[4 * c + 1] += x * v[k][c].y;
        acc[4 * c + 2] += x * v[k][c].z, acc[4 * c + 3] += x * v[k][c].w;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < L / 128; ++c)
    reinterpret_cast<float4*>(acc_s[warp])[32 * c + lane] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
  if (lane == 0) l_s[warp] = l;
  __syncthreads();
  const int64_t row = (int64_t)b * p.chunk * p.hq + (int64_t)rt * kLRows + r;
  l = (l_s[0] + l_s[1]) + (l_s[2] + l_s[3]);
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
  for (int c = threadIdx.x; c < L; c += 128) {
    const float x = ((acc_s[0][c] + acc_s[1][c]) + (acc_s[2][c] + acc_s[3][c])) * f;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[row * L + c] = __float2bfloat16_rn(x);
    else
      static_cast<float*>(p.out)[row * L + c] = x;
  }
}

// How a call is cut: row tiles per sequence, CTAs, and CTAs per row tile (0: a unit
// per CTA).  Sharing the positions costs the join, but fills the SMs where there are
// few units; it is taken where it leaves fewer of them idle.
struct LatentCut {
  int64_t tpb, ctas;
  int groups;
};
LatentCut latent_cut(int32_t batch, int32_t hq, int32_t chunk, int sms) {
  LatentCut c;
  c.tpb = ((int64_t)chunk * hq + kLRows - 1) / kLRows;
  const int64_t units = c.tpb * batch;
  const int64_t waves = (units + sms - 1) / sms;
  const double alone = (double)units / (double)(waves * sms);
  const int64_t groups = sms / c.tpb;
  const double shared = (double)(groups * c.tpb) / sms;
  if (groups > 1 && shared > alone) {
    c.groups = (int)groups;
    c.ctas = groups * c.tpb;
  } else {
    c.groups = 0;
    c.ctas = units < sms ? units : sms;
  }
  return c;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct LatentWorkspace {
  size_t rec, lse, o, bytes;
  LatentWorkspace(const LatentCut& c, int32_t batch, int32_t L) : rec(0), lse(0), o(0), bytes(16) {
    if (c.groups == 0) return;
    lse = align256((size_t)batch * c.tpb * sizeof(int2));
    o = lse + align256((size_t)c.ctas * 2 * kLRows * sizeof(float));
    bytes = o + (size_t)c.ctas * 2 * kLRows * L * sizeof(float);
  }
};

template <int L, int R>
kvq_status launch_latent(const LatentAttnParams& p, const LatentCut& cut, cudaStream_t s) {
  static DeviceOnce attr_set;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
  if (attr_set.pending(dev)) {
    if (cudaFuncSetAttribute(latent_attn_kernel<L, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, LGeo<L, R>::kBytes) !=
        cudaSuccess)
      return KVQ_ERR_CUDA;
    attr_set.mark(dev);
  }
  latent_attn_kernel<L, R><<<(unsigned)cut.ctas, kLThreads, LGeo<L, R>::kBytes, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
  if (cut.groups == 0) return KVQ_OK;
  const int rows = (int)((int64_t)p.chunk * p.hq < kLRows ? (int64_t)p.chunk * p.hq : kLRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * p.tpb * rows));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<L>, p, rows) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

bool latent_sizes_ok(int32_t batch, int32_t hq, int32_t chunk) {
  return (double)batch * ((double)chunk * hq + kLRows) <= (double)(1 << 30);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_latent_attn_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t latent_dim,
                                                  int32_t chunk) {
  if (batch < 1 || num_q_heads < 1 || chunk < 1 || !latent_dims_ok(16, latent_dim, 64) ||
      !latent_sizes_ok(batch, num_q_heads, chunk))
    return 0;
  const int sms = device_sm_count();
  return LatentWorkspace(latent_cut(batch, num_q_heads, chunk, sms > 0 ? sms : 148), batch, latent_dim).bytes;
}

extern "C" kvq_status kvq_latent_attn(const kvq_latent_cache* cache, int32_t batch, int32_t num_q_heads, int32_t chunk,
                                      const int32_t* d_seq_lens, const int32_t* d_chunk_lens, const void* q,
                                      float softmax_scale, void* out, int32_t out_dtype, void* workspace,
                                      size_t workspace_bytes, int32_t* d_err_flag, kvq_stream stream) {
  if (batch < 0 || num_q_heads < 1 || chunk < 0 || !(softmax_scale > 0.0f) || !(softmax_scale < 2.0e38f) ||
      (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_status st = check_latent_cache(cache, batch);
  if (st != KVQ_OK) return st;
  if (batch == 0 || chunk == 0) return KVQ_OK;
  if (d_seq_lens == nullptr || q == nullptr || out == nullptr || workspace == nullptr || !aligned_to(q, 16) ||
      !aligned_to(out, 16) || !aligned_to(workspace, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!latent_sizes_ok(batch, num_q_heads, chunk)) return KVQ_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  const LatentCut cut = latent_cut(batch, num_q_heads, chunk, sms > 0 ? sms : 148);
  const LatentWorkspace ws(cut, batch, cache->latent_dim);
  if (workspace_bytes < ws.bytes) return KVQ_ERR_WORKSPACE;
  if (sms <= 0) return KVQ_ERR_CUDA;
  LatentAttnParams p = {};
  p.c = *cache;
  p.lens = d_seq_lens, p.chunk_lens = d_chunk_lens;
  p.q = static_cast<const uint16_t*>(q), p.out = out, p.flag = d_err_flag;
  p.batch = batch, p.hq = num_q_heads, p.chunk = chunk, p.out_bf16 = out_dtype == KVQ_DTYPE_BF16;
  p.tpb = (int32_t)cut.tpb, p.groups = cut.groups;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.wait_ns = test_wait_limit_ns();
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.rec = reinterpret_cast<int2*>(w + ws.rec);
  p.part_lse = reinterpret_cast<float*>(w + ws.lse);
  p.part_o = reinterpret_cast<float*>(w + ws.o);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->rope_dim == 64) {
    if (cache->latent_dim == 512) return launch_latent<512, 64>(p, cut, s);
    if (cache->latent_dim == 256) return launch_latent<256, 64>(p, cut, s);
    return launch_latent<128, 64>(p, cut, s);
  }
  if (cache->latent_dim == 512) return launch_latent<512, 32>(p, cut, s);
  if (cache->latent_dim == 256) return launch_latent<256, 32>(p, cut, s);
  return launch_latent<128, 32>(p, cut, s);
}
