// The bounded waits of csrc/diff.cuh on barriers that nothing arrives at: one CTA of two
// warps, each wait with a limit.  Per wait: whether it was satisfied, and its time in ns.
#include "diff.cuh"

__global__ void wait_probe(uint64_t limit_ns, uint64_t* out) {
  __shared__ uint64_t bar[2];
  if (threadIdx.x == 0) {
    salad::mbar_init(&bar[0], 1);
    salad::mbar_init(&bar[1], 1);
    salad::fence_mbar_init();
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {  // a warp: the wait that runs out, then a later one
    bool ok = limit_ns != 0;
    const uint32_t polls = salad::polls_of(limit_ns);
    for (int i = 0; i < 2; ++i) {
      const uint64_t t0 = salad::global_timer_ns();
      salad::mbar_await(&bar[0], 0, polls, ok);
      if (lane == 0) out[2 * i] = ok, out[2 * i + 1] = salad::global_timer_ns() - t0;
    }
  } else if (lane == 0) {  // one thread
    const uint64_t t0 = salad::global_timer_ns();
    const bool ok = salad::mbar_await_one(&bar[1], 0, limit_ns);
    out[4] = ok, out[5] = salad::global_timer_ns() - t0;
  }
}

extern "C" int wait_probe_run(uint64_t limit_ns, uint64_t* out) {
  wait_probe<<<1, 64>>>(limit_ns, out);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? (int)e : (int)cudaDeviceSynchronize();
}
