// Rotary positions of q and k (and, with the sine negated, their gradients).
// A head's first `rot` features hold rot/2 pairs; pair i of a token at position
// p (of the pair's axis) turns by the angle p f_i:
//   y1 = m (x1 cos - x2 sin),   y2 = m (x2 cos + x1 sin)
// The rotation is orthogonal, so its gradient is the turn by the opposite angle
// times the same m.  Features from `rot` on are copied.
//
// Bound by memory: each value is read once and written once (6 flops a pair).
// One warp takes one token and a run of its heads: the angles of a token serve
// all of its heads, so the warp forms them once (two pairs a lane at rot = 128),
// leaves cos and sin in its own piece of shared memory and keeps the eight pairs
// that a lane works on in registers for every head.  The product p f and its
// reduction to [-1, 1] half turns are in fp64 (at p = 2^31 the angle is still
// good to 2^-22), sine and cosine of the reduced angle in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"

namespace salad {
namespace {

constexpr int kRopeWarps = 4;  // (8: 70.1 us at 32,760 tokens x 24 heads of 128, 4: 68.3)

template <typename T>
struct Raw8;  // eight consecutive values as loaded and stored
template <>
struct Raw8<float> {
  float4 a, b;
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Raw8<__half> {
  uint4 a;
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    r.a = __ldcs(reinterpret_cast<const float4*>(p));
    r.b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  } else {
    r.a = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  return r;
}
__device__ __forceinline__ void widen(const Raw8<float>& r, float (&v)[8]) {
  v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
  v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
__device__ __forceinline__ void widen(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void widen(const Raw8<__half>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

// The position of token n of sequence b along an axis.
__device__ __forceinline__ int rope_position(const RopeArgs& a, int b, int n, int axis) {
  if (a.positions != nullptr) return a.positions[b * a.pos_stride_b + (int64_t)n * a.axes + axis];
  const int t = n / a.grid_w;  // (frame, row) index
  if (axis == 0) return a.origin[0] + t / a.grid_h;
  if (axis == 1) return a.origin[1] + t % a.grid_h;
  return a.origin[2] + n % a.grid_w;
}

// m cos and m sin of every pair of a token, by the lanes of one warp.
__device__ __forceinline__ void warp_angles(const RopeArgs& a, int b, int n, int lane, float2* cs) {
  int pos[3];
#pragma unroll
  for (int x = 0; x < 3; ++x) pos[x] = x < a.axes ? rope_position(a, b, n, x) : 0;
  for (int i = lane; i < a.rot / 2; i += 32) {
    const int p = i < a.axis_end[0] ? pos[0] : i < a.axis_end[1] ? pos[1] : pos[2];
    const double u = (double)p * a.inv_freq[i] * 0.31830988618379067154;  // half turns
    float s, c;
    sincospif((float)(u - 2.0 * rint(0.5 * u)), &s, &c);
    cs[i] = make_float2(a.scale * c, (a.inverse ? -a.scale : a.scale) * s);
  }
  __syncwarp();
}

// A lane works on eight pairs of a head: pairs 8u .. 8u + 7 lie in two runs of
// eight features, [8u, +8) and [rot/2 + 8u, +8) in the half layout, [16u, +16)
// in the interleaved one; behind rot a lane copies 16 features.
template <typename X, typename Y>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const RopeArgs a) {
  extern __shared__ float2 rope_cs[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = (int64_t)blockIdx.x * kRopeWarps + warp;
  if (token >= (int64_t)a.B * a.N) return;
  const int b = (int)(token / a.N), n = (int)(token % a.N);
  float2* cs = rope_cs + warp * (a.rot / 2);
  warp_angles(a, b, n, lane, cs);

  const int upt = a.d / 16, slots = 32 / upt;  // lanes a head takes, heads a warp takes at once
  const int u = lane % upt, slot = lane / upt;
  if (slot >= slots) return;
  const bool turn = 16 * u < a.rot;
  const int o1 = turn && !a.interleaved ? 8 * u : 16 * u;
  const int o2 = turn && !a.interleaved ? a.rot / 2 + 8 * u : 16 * u + 8;
  float c[8], s[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 w = reinterpret_cast<const float4*>(cs)[4 * u + i / 2];
      c[i] = w.x, s[i] = w.y, c[i + 1] = w.z, s[i + 1] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  }
  const int heads = a.t[0].heads + a.t[1].heads, first = blockIdx.y * a.heads_per_warp;
  const int end = min(heads, first + a.heads_per_warp);
  auto row = [&](int h, const X*& x, Y*& y) {
    const bool second = h >= a.t[0].heads;
    const RopeTensor& t = a.t[second ? 1 : 0];
    const int hh = second ? h - a.t[0].heads : h;
    x = static_cast<const X*>(t.x) + b * t.xb + n * t.xn + hh * t.xh;
    y = static_cast<Y*>(t.y) + b * t.yb + n * t.yn + hh * t.yh;
  };
  constexpr int kDeep = 3;  // heads in flight a lane (2: 74.5 us, 6: 78.3)
  for (int h0 = first + slot; h0 < end; h0 += kDeep * slots) {
    Raw8<X> r1[kDeep], r2[kDeep];
    Y* dst[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int h = h0 + k * slots;
      if (h < end) {
        const X* x;
        row(h, x, dst[k]);
        r1[k] = load8(x + o1);
        r2[k] = load8(x + o2);
      }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      if (h0 + k * slots >= end) break;
      float v1[8], v2[8], w1[8], w2[8];
      widen(r1[k], v1);
      widen(r2[k], v2);
      if (!turn) {
        store8(dst[k] + o1, v1);
        store8(dst[k] + o2, v2);
        continue;
      }
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w1[2 * i] = fmaf(v1[2 * i], c[i], -v1[2 * i + 1] * s[i]);
          w1[2 * i + 1] = fmaf(v1[2 * i + 1], c[i], v1[2 * i] * s[i]);
          w2[2 * i] = fmaf(v2[2 * i], c[4 + i], -v2[2 * i + 1] * s[4 + i]);
          w2[2 * i + 1] = fmaf(v2[2 * i + 1], c[4 + i], v2[2 * i] * s[4 + i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w1[i] = fmaf(v1[i], c[i], -v2[i] * s[i]);
          w2[i] = fmaf(v2[i], c[i], v1[i] * s[i]);
        }
      }
      store8(dst[k] + o1, w1);
      store8(dst[k] + o2, w2);
    }
  }
}

// Any width, part and alignment: one lane a pair (or a feature behind rot).
template <typename X, typename Y>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_any_kernel(const RopeArgs a) {
  extern __shared__ float2 rope_cs[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = (int64_t)blockIdx.x * kRopeWarps + warp;
  if (token >= (int64_t)a.B * a.N) return;
  const int b = (int)(token / a.N), n = (int)(token % a.N);
  float2* cs = rope_cs + warp * (a.rot / 2);
  warp_angles(a, b, n, lane, cs);
  const int heads = a.t[0].heads + a.t[1].heads, first = blockIdx.y * a.heads_per_warp;
  const int end = min(heads, first + a.heads_per_warp), half = a.rot / 2, items = half + a.d - a.rot;
  for (int h = first; h < end; ++h) {
    const bool second = h >= a.t[0].heads;
    const RopeTensor& t = a.t[second ? 1 : 0];
    const int hh = second ? h - a.t[0].heads : h;
    const X* x = static_cast<const X*>(t.x) + b * t.xb + n * t.xn + hh * t.xh;
    Y* y = static_cast<Y*>(t.y) + b * t.yb + n * t.yn + hh * t.yh;
    for (int i = lane; i < items; i += 32) {
      if (i >= half) {
        const int e = a.rot + i - half;
        put(y + e, to_f32(x[e]));
        continue;
      }
      const int e1 = a.interleaved ? 2 * i : i, e2 = a.interleaved ? 2 * i + 1 : half + i;
      const float v1 = to_f32(x[e1]), v2 = to_f32(x[e2]);
      put(y + e1, fmaf(v1, cs[i].x, -v2 * cs[i].y));
      put(y + e2, fmaf(v2, cs[i].x, v1 * cs[i].y));
    }
  }
}

template <typename X, typename Y>
cudaError_t launch_rope_t(RopeArgs a, cudaStream_t s) {
  const int64_t tokens = (int64_t)a.B * a.N;
  const int heads = a.t[0].heads + a.t[1].heads;
  // Few tokens (a sampling step): a token's heads are shared out over more
  // warps, down to the heads a warp takes at once, until there are 16 warps an
  // SM; with many tokens one warp takes all heads and forms the angles once.
  const int slots = a.wide ? 32 / (a.d / 16) : 1;
  const int64_t want = (148 * 16 + tokens - 1) / tokens;
  const int64_t groups = std::max<int64_t>(1, (heads + slots - 1) / slots);
  const int64_t shares = std::max<int64_t>(1, std::min(want, groups));
  a.heads_per_warp = (int)((groups + shares - 1) / shares) * slots;
  const dim3 grid((unsigned)((tokens + kRopeWarps - 1) / kRopeWarps),
                  (unsigned)((heads + a.heads_per_warp - 1) / a.heads_per_warp));
  const size_t smem = (size_t)kRopeWarps * (a.rot / 2) * sizeof(float2);
  if (a.wide)
    rope_kernel<X, Y><<<grid, 32 * kRopeWarps, smem, s>>>(a);
  else
    rope_any_kernel<X, Y><<<grid, 32 * kRopeWarps, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename X>
cudaError_t launch_rope_x(const RopeArgs& a, int y_type, cudaStream_t s) {
  if (y_type == SALAD_F32) return launch_rope_t<X, float>(a, s);
  if (y_type == SALAD_BF16) return launch_rope_t<X, __nv_bfloat16>(a, s);
  return launch_rope_t<X, __half>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int x_type, int y_type, cudaStream_t s) {
  if (x_type == SALAD_F32) return launch_rope_x<float>(a, y_type, s);
  if (x_type == SALAD_BF16) return launch_rope_x<__nv_bfloat16>(a, y_type, s);
  return launch_rope_x<__half>(a, y_type, s);
}

}  // namespace salad
