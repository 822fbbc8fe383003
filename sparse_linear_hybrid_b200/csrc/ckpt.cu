// Activation checkpoints in 8 bits.  A row's values are taken in groups of 32;
// a group keeps one byte e + 127 and a code a value:
//   e    = the smallest exponent >= -127 with max|x| / 2^e <= 127 (int8) or 448 (e4m3)
//   code = round to nearest even (x / 2^e),   decoded = code 2^e
// Scales are powers of two, so x / 2^e is exact in fp32, the code depends on x
// alone (not on the order or width of the arithmetic) and the decoded value has
// at most 7 (int8) or 4 (e4m3) significant bits: exact in bf16 (from 2^-133 on).  A group that
// holds an infinity or a NaN has the byte 255 and decodes to NaN.
//
// Bound by memory: 2 + 1 + 1/32 bytes a bf16 value each way (three tensors of 50 M
// values packed and unpacked again: 148 us, 6.2 TB/s).  A lane takes 16 values (two
// 16-byte loads of bf16, one 16-byte store of codes), two lanes a group; more
// pieces a lane were slower (two 153 us, four 157).  Rounding to int8 adds 1.5 2^23 (the
// fused multiply-add rounds to an integer that sits in the low byte), so no
// conversion instruction is needed on that side.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"

namespace salad {
namespace {

constexpr int kCkptThreads = 256;
constexpr float kRound = 12582912.f;  // 1.5 * 2^23

__device__ __forceinline__ float f32_of(float x) { return x; }
__device__ __forceinline__ float f32_of(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float f32_of(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

template <typename T>
__device__ __forceinline__ void load16(const T* p, uint4 (&r)[sizeof(T)]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) r[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
}
__device__ __forceinline__ void widen(const uint4 (&r)[4], float (&v)[16], float) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = __uint_as_float(r[i].x), v[4 * i + 1] = __uint_as_float(r[i].y);
    v[4 * i + 2] = __uint_as_float(r[i].z), v[4 * i + 3] = __uint_as_float(r[i].w);
  }
}
__device__ __forceinline__ void widen(const uint4 (&r)[2], float (&v)[16], __nv_bfloat16) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void widen(const uint4 (&r)[2], float (&v)[16], __half) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[8 * i + 2 * j] = f.x;
      v[8 * i + 2 * j + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
}
__device__ __forceinline__ uint32_t pair_bits(float x, float y, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pair_bits(float x, float y, __half) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pair_bits(v[8 * i + 2 * j], v[8 * i + 2 * j + 1], T{});
    __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// The scale byte of a group from the bits of its largest magnitude: the
// exponent of the leading bit less that of the largest code, one more where the
// mantissa lies above the largest code's.
template <bool FP8>
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255;
  const int field = (int)(amax_bits >> 23);
  const uint32_t mant = amax_bits & 0x7FFFFFu;
  const int e = FP8 ? field - 8 + (mant > 0x600000u) : field - 6 + (mant > 0x7E0000u);  // 448 = 1.75 2^8, 127 = 1.984375 2^6
  return max(e, 0);
}
// 2^-(byte - 127); 0 for the byte of a group without a scale.
__device__ __forceinline__ float inverse_scale(int byte) {
  return byte == 255 ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);
}
// 2^(byte - 127), NaN for 255 (2^-127 is a subnormal).
__device__ __forceinline__ float scale_of(int byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : (uint32_t)byte << 23);
}

// Codes of four values (a group without a scale has codes 0: its infinities and
// NaNs do not reach the conversion).
template <bool FP8>
__device__ __forceinline__ uint32_t encode4(const float* v, float inv) {
  if constexpr (FP8) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  } else {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(v[i], inv, kRound));
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
}
template <bool FP8>
__device__ __forceinline__ void decode4(uint32_t codes, float scale, float* v) {
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> 16 * i & 0xFFFFu), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  } else {
    const uint32_t u = codes ^ 0x80808080u;  // code + 128 in the low byte of 2^23's mantissa
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (__uint_as_float(0x4B000000u | (u >> 8 * i & 0xFFu)) - 8388736.f) * scale;
  }
}

// The largest finite value of a type, and the smallest scale byte from which a
// decoded value can pass it (the largest value of a group may round up).
template <typename T>
struct Top;
template <>
struct Top<float> {
  static constexpr float value = 3.402823466e38f;
  static constexpr int byte = 239;
};
template <>
struct Top<__nv_bfloat16> {
  static constexpr float value = 3.389531390e38f;
  static constexpr int byte = 239;
};
template <>
struct Top<__half> {
  static constexpr float value = 65504.f;
  static constexpr int byte = 127;
};
template <typename T>
__device__ __forceinline__ float capped(float x, int byte) {
  return byte == 255 ? __uint_as_float(0x7FC00000u) : fminf(fmaxf(x, -Top<T>::value), Top<T>::value);
}

// 16 values a lane; cols is a multiple of 32 and every row starts on 16 bytes.
template <typename T, bool FP8>
__global__ void __launch_bounds__(kCkptThreads) ckpt_pack_kernel(const CkptArgs a) {
  const CkptPart& p = a.part[blockIdx.y];
  const T* x = static_cast<const T*>(p.x);
  const uint32_t per_row = (uint32_t)(a.cols / 16), total = (uint32_t)a.rows * per_row;
  const uint32_t id = blockIdx.x * kCkptThreads + threadIdx.x;
  float v[16];
  uint32_t top = 0;
  if (id < total) {
    uint4 raw[sizeof(T)];
    const uint32_t row = a.one_row ? 0u : id / per_row;
    load16(x + (int64_t)row * p.stride + (int64_t)(id - row * per_row) * 16, raw);
    widen(raw, v, T{});
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  if (id >= total) return;
  const int byte = scale_byte<FP8>(top);
  const float inv = inverse_scale(byte);
  uint4 c = make_uint4(0u, 0u, 0u, 0u);
  if (byte != 255)
    c = make_uint4(encode4<FP8>(v, inv), encode4<FP8>(v + 4, inv), encode4<FP8>(v + 8, inv), encode4<FP8>(v + 12, inv));
  __stcs(reinterpret_cast<uint4*>(p.codes) + id, c);
  if ((threadIdx.x & 1) == 0) p.scales[id / 2] = (uint8_t)byte;
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(kCkptThreads) ckpt_unpack_kernel(const CkptArgs a) {
  const CkptPart& p = a.part[blockIdx.y];
  T* y = static_cast<T*>(p.y);
  const uint32_t per_row = (uint32_t)(a.cols / 16), total = (uint32_t)a.rows * per_row;
  const uint32_t id = blockIdx.x * kCkptThreads + threadIdx.x;
  if (id >= total) return;
  const uint4 c = __ldcs(reinterpret_cast<const uint4*>(p.codes) + id);
  const int byte = p.scales[id / 2];
  const float scale = scale_of(byte);
  float v[16];
  decode4<FP8>(c.x, scale, v);
  decode4<FP8>(c.y, scale, v + 4);
  decode4<FP8>(c.z, scale, v + 8);
  decode4<FP8>(c.w, scale, v + 12);
  if (byte >= Top<T>::byte) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = capped<T>(v[i], byte);
  }
  const uint32_t row = a.one_row ? 0u : id / per_row;
  store16(y + (int64_t)row * p.stride + (int64_t)(id - row * per_row) * 16, v);
}

// Any width and alignment: one warp a group, one lane a value.
template <typename T, bool FP8>
__global__ void __launch_bounds__(kCkptThreads) ckpt_pack_any_kernel(const CkptArgs a) {
  const CkptPart& p = a.part[blockIdx.y];
  const uint32_t lane = threadIdx.x & 31, groups = (uint32_t)((a.cols + 31) / 32);
  const uint32_t id = blockIdx.x * (kCkptThreads / 32) + (threadIdx.x >> 5);
  if (id >= (uint32_t)a.rows * groups) return;
  const uint32_t row = id / groups, col = (id - row * groups) * 32 + lane;
  float v = 0.f;
  if (col < (uint32_t)a.cols) v = f32_of(static_cast<const T*>(p.x)[(int64_t)row * p.stride + col]);
  const int byte = scale_byte<FP8>(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
  const float w[4] = {byte == 255 ? 0.f : v, 0.f, 0.f, 0.f};
  if (col < (uint32_t)a.cols)
    p.codes[(int64_t)row * a.cols + col] = (uint8_t)encode4<FP8>(w, inverse_scale(byte));
  if (lane == 0) p.scales[id] = (uint8_t)byte;
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(kCkptThreads) ckpt_unpack_any_kernel(const CkptArgs a) {
  const CkptPart& p = a.part[blockIdx.y];
  const uint32_t lane = threadIdx.x & 31, groups = (uint32_t)((a.cols + 31) / 32);
  const uint32_t id = blockIdx.x * (kCkptThreads / 32) + (threadIdx.x >> 5);
  if (id >= (uint32_t)a.rows * groups) return;
  const uint32_t row = id / groups, col = (id - row * groups) * 32 + lane;
  if (col >= (uint32_t)a.cols) return;
  const int byte = p.scales[id];
  float v[4];
  decode4<FP8>(p.codes[(int64_t)row * a.cols + col], scale_of(byte), v);
  put(static_cast<T*>(p.y) + (int64_t)row * p.stride + col, capped<T>(v[0], byte));
}

template <typename T, bool FP8>
cudaError_t launch_ckpt_t(const CkptArgs& a, bool pack, cudaStream_t s) {
  const uint64_t per_cta = a.wide ? (uint64_t)kCkptThreads : kCkptThreads / 32;
  const uint64_t units = (uint64_t)a.rows * (a.wide ? a.cols / 16 : (a.cols + 31) / 32);
  const dim3 grid((unsigned)((units + per_cta - 1) / per_cta), (unsigned)a.parts);
  if (pack && a.wide)
    ckpt_pack_kernel<T, FP8><<<grid, kCkptThreads, 0, s>>>(a);
  else if (pack)
    ckpt_pack_any_kernel<T, FP8><<<grid, kCkptThreads, 0, s>>>(a);
  else if (a.wide)
    ckpt_unpack_kernel<T, FP8><<<grid, kCkptThreads, 0, s>>>(a);
  else
    ckpt_unpack_any_kernel<T, FP8><<<grid, kCkptThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// dq, dk and dv in bf16 from their fp32 sums.
__global__ void __launch_bounds__(256) narrow_kernel(const float* __restrict__ x, uint16_t* __restrict__ y0,
                                                     uint16_t* __restrict__ y1, uint16_t* __restrict__ y2,
                                                     int64_t count8) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= count8) return;
  const float4* src = reinterpret_cast<const float4*>(x) + ((int64_t)blockIdx.y * count8 + i) * 2;
  const float4 a = __ldcs(src), b = __ldcs(src + 1);
  uint16_t* y = blockIdx.y == 0 ? y0 : blockIdx.y == 1 ? y1 : y2;
  reinterpret_cast<uint4*>(y)[i] =
      make_uint4(pair_bits(a.x, a.y, __nv_bfloat16{}), pair_bits(a.z, a.w, __nv_bfloat16{}),
                 pair_bits(b.x, b.y, __nv_bfloat16{}), pair_bits(b.z, b.w, __nv_bfloat16{}));
}

}  // namespace

cudaError_t launch_ckpt(const CkptArgs& a, bool pack, int type, bool fp8, cudaStream_t s) {
  if (type == SALAD_F32) return fp8 ? launch_ckpt_t<float, true>(a, pack, s) : launch_ckpt_t<float, false>(a, pack, s);
  if (type == SALAD_BF16)
    return fp8 ? launch_ckpt_t<__nv_bfloat16, true>(a, pack, s) : launch_ckpt_t<__nv_bfloat16, false>(a, pack, s);
  return fp8 ? launch_ckpt_t<__half, true>(a, pack, s) : launch_ckpt_t<__half, false>(a, pack, s);
}

cudaError_t launch_narrow3(const float* x, uint16_t* y0, uint16_t* y1, uint16_t* y2, int64_t count, cudaStream_t s) {
  const dim3 grid((unsigned)((count / 8 + 255) / 256), 3);
  narrow_kernel<<<grid, 256, 0, s>>>(x, y0, y1, y2, count / 8);
  return cudaGetLastError();
}

}  // namespace salad
