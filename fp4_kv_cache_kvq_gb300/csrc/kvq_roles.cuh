// kvq_roles.cuh -- what kernels whose warps have roles of their own share: bounded
// waits of a warp, the issuing lane, and packed fp32 arithmetic.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

// A wait of the whole warp with one outcome; it gives up after the library's limit
// (or a test's, which polls: a suspending wait could outlast it), or with any other
// wait of the CTA.
struct BoundedWaits {
  volatile int* abort;
  uint64_t limit;  // a test's, ns, or 0
  // whether the phase is over; does not wait
  __device__ __forceinline__ bool over(uint32_t bar, uint32_t parity) const { return mbar_test_wait(bar, parity); }
  // (suspended in the barrier: a warp that polls takes issue slots from those that work)
  __device__ __forceinline__ bool look(uint32_t bar, uint32_t parity) const {
    return limit ? mbar_test_wait(bar, parity) : mbar_try_wait_hint(bar, parity, 1000000u);
  }
  __device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity) const {
    if (look(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (true) {
      if (look(bar, parity)) return true;
      if (*abort) return false;
      if (global_ns() - t0 > (limit ? limit : kWaitLimitNs)) {
        *abort = 1;
        return false;
      }
    }
  }
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity))) return true;
    return __all_sync(0xFFFFFFFFu, lane_wait(bar, parity));
  }
};

// One lane of a converged warp.  (A lane picked by its number makes the compiler treat
// the descriptors as different from lane to lane: 70 cycles an MMA.)
__device__ __forceinline__ bool elect_one_of_warp() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Two fp32 values side by side.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

}  // namespace kvq
