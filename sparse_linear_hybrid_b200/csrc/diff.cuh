// What the two differential kernels' files share beside ptx.cuh: waits and issuing by
// converged warps, and a few arithmetic instructions.
#pragma once

#include "ptx.cuh"

namespace salad {

__device__ __forceinline__ float lambda_of(const void* lam, int bf16, int h) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(lam)[h] << 16) : static_cast<const float*>(lam)[h];
}

// A value that is the same in all lanes of a converged warp, told to the compiler
// (it then keeps what follows from it in uniform registers and branches as a warp).
__device__ __forceinline__ int warp_uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// True once the phase with the given parity has completed; one look, where
// mbar_try_wait may hold the thread for a while.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait of a converged warp, lane by lane: after `polls` polls a lane's `ok` turns
// false, and its later waits only look.  The polls behind the first do not block
// (mbar_try_wait held a thread for 4 us) and sleep 40 ns at most, so that each takes
// 128 ns or less (64 measured) and their count keeps the limit in time; reading the timer
// in their place cost the differential forward 2 to 6 %.  The caller goes on with its
// loop, without a vote or a way out (either costs the compiler its uniform branches:
// 1,051 against 955 us for the differential forward at 1.3B), but a lane arrives,
// commits and issues nothing while its ok is false: a stage given back before its copy
// has landed would let the CTA end with the copy in flight.  The caller votes on ok
// behind its loop.  With a limit of 0 (a test hook) ok is false from the start.
__device__ __forceinline__ uint32_t polls_of(uint64_t limit_ns) {
  const uint64_t n = limit_ns / 128;
  return n > 0x7FFFFFFFull ? 0x7FFFFFFFu : (uint32_t)n + 1u;
}
__device__ __forceinline__ void mbar_await(uint64_t* bar, uint32_t parity, uint32_t polls, bool& ok) {
  if (!mbar_try_wait(bar, parity)) {
    uint32_t left = ok ? polls : 1u;
#pragma unroll 1
    do {
      if (--left == 0) {
        ok = false;
        break;
      }
      __nanosleep(20);
    } while (!mbar_test_wait(bar, parity));
  }
  __syncwarp();
}
// Bounded wait of one thread that has time (a producer some stages ahead).
__device__ __forceinline__ bool mbar_await_one(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  if (limit_ns == 0) return false;
  const uint64_t t0 = global_timer_ns();
  do {
    __nanosleep(100);
    if (mbar_test_wait(bar, parity)) return true;
  } while (global_timer_ns() - t0 < limit_ns);
  return false;
}

// True in one lane of a converged warp, always the same one.  An issuing warp
// that runs its loop as a whole and branches on this only around the products
// keeps their descriptors in uniform registers; a single thread that runs the
// loop (lane == 0) moves them there for every product: 128 x 64 x 16 products
// from tensor memory issue every 33 cycles this way and every 55 the other,
// 16 alternating ones from shared and tensor memory in 1,040 against 1,980.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// fmax3, NaN when one of them is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace salad
