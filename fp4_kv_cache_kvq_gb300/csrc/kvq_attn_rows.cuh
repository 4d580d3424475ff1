// kvq_attn_rows.cuh -- attention of 16 query rows per CTA over tiles of 32
// positions in fp32 (scores and sums by plain FMAs): one pass with the running
// maximum and sum of the softmax.  Src hands over the rows of queries, keys and
// values; it serves the latent cache and dense keys and values alike.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

constexpr int kRowsR = 16, kPosR = 32, kThreadsR = 256;

struct RowsShape {
  int dk, dv;  // widths of a score and of a value
  __host__ __device__ int kpad() const { return dk + 1; }
  __host__ __device__ size_t bytes() const {
    return sizeof(float) * ((size_t)kRowsR * dk + (size_t)kPosR * kpad() + (size_t)kPosR * dv + kRowsR * kPosR + 3 * kRowsR);
  }
};

// Rows r < rows of one unit; row r attends positions 0 .. src.last(r); positions
// up to `limit` are visited.  src.query(r, c), src.load(pos, ks, vs) (thread-wide
// copy of one position's key and value into shared memory), src.store(r, c, x).
template <typename Src>
__device__ void attend_rows(const Src& src, const RowsShape sh, int rows, int64_t limit, float scale_log2, float* sm) {
  float* q = sm;
  float* ks = q + kRowsR * sh.dk;
  float* vs = ks + kPosR * sh.kpad();
  float* p = vs + kPosR * sh.dv;
  float* mx = p + kRowsR * kPosR;
  float* sum = mx + kRowsR;
  float* fac = sum + kRowsR;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kRowsR * sh.dk; i += kThreadsR) {
    const int r = i / sh.dk;
    q[i] = r < rows ? src.query(r, i % sh.dk) : 0.0f;
  }
  if (tid < kRowsR) mx[tid] = -INFINITY, sum[tid] = 0.0f;
  float acc[kRowsR][2];
#pragma unroll
  for (int r = 0; r < kRowsR; ++r) acc[r][0] = acc[r][1] = 0.0f;
  for (int64_t p0 = 0; p0 < limit; p0 += kPosR) {
    __syncthreads();
    for (int j = warp; j < kPosR; j += kThreadsR / 32)
      src.load(p0 + j < limit ? p0 + j : -1, ks + j * sh.kpad(), vs + j * sh.dv, lane);
    __syncthreads();
    for (int i = tid; i < kRowsR * kPosR; i += kThreadsR) {  // a warp per row: the row's scores in its lanes
      const int r = i / kPosR, j = i % kPosR;
      const float* a = q + r * sh.dk;
      const float* b = ks + j * sh.kpad();
      float s = 0.0f;
      for (int c = 0; c < sh.dk; ++c) s = fmaf(a[c], b[c], s);
      const bool in = r < rows && src.attends(p0 + j) && p0 + j <= src.last(r);
      s = in ? s * scale_log2 : -INFINITY;
      float m = s;
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float old = mx[r], top = fmaxf(old, m), ref = top == -INFINITY ? 0.0f : top;
      const float e = exp2f(s - ref);
      float l = e;
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      p[i] = e;
      __syncwarp();
      if (lane == 0) {
        const float f = exp2f(old - ref);
        fac[r] = f;
        sum[r] = sum[r] * f + l;
        mx[r] = top;
      }
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
      const int c = tid + k * kThreadsR;
      if (c >= sh.dv) continue;
#pragma unroll
      for (int r = 0; r < kRowsR; ++r) {
        float o = acc[r][k] * fac[r];
        for (int j = 0; j < kPosR; ++j) {
          const float w = p[r * kPosR + j];
          if (w != 0.0f) o = fmaf(w, vs[j * sh.dv + c], o);
        }
        acc[r][k] = o;
      }
    }
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    const int c = tid + k * kThreadsR;
    if (c >= sh.dv) continue;
#pragma unroll
    for (int r = 0; r < kRowsR; ++r)
      if (r < rows) src.store(r, c, sum[r] == 0.0f ? 0.0f : acc[r][k] / sum[r]);
  }
}

}  // namespace kvq
