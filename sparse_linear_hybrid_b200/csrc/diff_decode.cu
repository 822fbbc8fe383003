// Differential attention (diff.cu) of a few query rows, one in general, against a
// cache of keys and values: query i of sequence b sees keys [0, lens[b]) (0 keys:
// the output is 0).
//
// Bound by memory: each live key and value is read once per query or pair of
// queries (12 heads of 128, one query each: 4 x 32,760 keys 145 us, 5.6 TB/s;
// 4 x 28,665 keys 128 us, 5.5 TB/s; lengths of 24,570 to 32,760 with that sum 133 us,
// because the split goes by the cache's capacity and the CTAs of the longest sequence
// have the most keys).  The keys of a (b, h) are split over the CTAs of a cluster (up
// to 16) so that a short batch still fills the machine; every warp keeps an online
// softmax of its keys (running maxima, sums and weighted values of both maps in fp32
// registers, d/8 lanes a key, eight features a lane), the warps join in
// shared memory and the cluster through distributed shared memory: one launch,
// no workspace.  Lanes of a key's first half of features form the score of map
// 1, the others that of map 2, and one exchange hands each the other's.
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace salad {
namespace {

namespace cg = cooperative_groups;

constexpr int kDecWarps = 8;
constexpr int kDecSplits = 16;

// A maximum over no key, or over scores of -inf alone.  It is finite, so that differences
// to it are never -inf - -inf: such a key weighs 2^-inf = 0 and such a part has l = 0.
constexpr float kDecNone = -3.402823466e38f;

// Joins (m, l, acc) of another part into this one.
template <int E>
__device__ __forceinline__ void join(float& m, float& l, float (&acc)[E], float m2, float l2, const float (&acc2)[E]) {
  const float top = fmaxf(m, m2);
  const float a = ex2_approx(m - top), b = ex2_approx(m2 - top);
  m = top;
  l = l * a + l2 * b;
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = acc[i] * a + acc2[i] * b;
}

__device__ __forceinline__ void widen8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo_to_f32(w[i]);
    v[2 * i + 1] = bf16_hi_to_f32(w[i]);
  }
}

// CTAs an SM, and keys a lane group works on at once (as many again are on their
// way): what keeps the registers within bounds without spills.
template <int NQ>
struct DecCfg {
  static constexpr int CTAS = 2;
  static constexpr int DEEP = NQ == 1 ? 3 : 1;
};

template <int D, int NQ>
__global__ void __launch_bounds__(32 * kDecWarps, DecCfg<NQ>::CTAS)
    diff_decode_kernel(const DiffDecodeArgs a, int splits) {
  constexpr int LPK = D / 8;          // lanes a key
  constexpr int KPW = 32 / LPK;       // keys a warp takes at once
  constexpr int DEEP = DecCfg<NQ>::DEEP;
  // per query and map: maximum, sum and weighted values of the warps, then of the CTA
  __shared__ float sm[NQ][2][kDecWarps], sl[NQ][2][kDecWarps];
  __shared__ __align__(16) float sacc[NQ][2][kDecWarps][D];
  __shared__ float cm[NQ][2], cl[NQ][2], cacc[NQ][2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % splits, bh = blockIdx.x / splits, b = bh / a.heads, h = bh % a.heads;
  const int q0 = blockIdx.y * NQ;
  const int part = lane % LPK, slot = lane / LPK;
  const int len = min(max(a.lens[b], 0), a.cap);
  // this CTA's keys [k0, k1): whole runs of KPW keys
  const int runs = (len + KPW - 1) / KPW, per = (runs + splits - 1) / splits;
  const int k0 = min(len, split * per * KPW), k1 = min(len, (split + 1) * per * KPW);

  float q[NQ][8];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (q0 + i < a.Nq)
      r = *reinterpret_cast<const uint4*>(a.q + (((int64_t)b * a.Nq + q0 + i) * a.heads + h) * D + part * 8);
    widen8(r, q[i]);
#pragma unroll
    for (int f = 0; f < 8; ++f) q[i][f] *= a.scale_log2;
  }
  float m1[NQ], m2[NQ], l1[NQ], l2[NQ], acc1[NQ][8], acc2[NQ][8];
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    m1[i] = m2[i] = kDecNone;
    l1[i] = l2[i] = 0.f;
#pragma unroll
    for (int f = 0; f < 8; ++f) acc1[i][f] = acc2[i][f] = 0.f;
  }
  const int64_t row = (int64_t)a.heads * D;
  const uint16_t* kp = a.k + (int64_t)b * a.cap * row + (int64_t)h * D + part * 8;
  const uint16_t* vp = a.v + (int64_t)b * a.cap * row + (int64_t)h * D + part * 8;
  const bool first = part < LPK / 2;
  constexpr int STEP = kDecWarps * KPW * DEEP;  // keys of the CTA an iteration
  auto fetch = [&](int base, uint4 (&kr)[DEEP], uint4 (&vr)[DEEP]) {
#pragma unroll
    for (int u = 0; u < DEEP; ++u) {
      const int key = base + u * kDecWarps * KPW + slot;
      kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
      if (key < k1) {
        kr[u] = __ldcs(reinterpret_cast<const uint4*>(kp + key * row));
        vr[u] = __ldcs(reinterpret_cast<const uint4*>(vp + key * row));
      }
    }
  };
  // the next iteration's keys and values are on their way while one is worked on
  uint4 kr[2][DEEP], vr[2][DEEP];
  fetch(k0 + warp * KPW, kr[0], vr[0]);
  auto work = [&](int base, const uint4 (&kr)[DEEP], const uint4 (&vr)[DEEP]) {
    bool live[DEEP];
#pragma unroll
    for (int u = 0; u < DEEP; ++u) live[u] = base + u * kDecWarps * KPW + slot < k1;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float s1[DEEP], s2[DEEP], t1 = m1[i], t2 = m2[i];
#pragma unroll
      for (int u = 0; u < DEEP; ++u) {
        float k8[8], s = 0.f;
        widen8(kr[u], k8);
#pragma unroll
        for (int f = 0; f < 8; ++f) s = fmaf(q[i][f], k8[f], s);
#pragma unroll
        for (int o = 1; o < LPK / 2; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float other = __shfl_xor_sync(0xffffffffu, s, LPK / 2);
        s1[u] = live[u] ? (first ? s : other) : -INFINITY;
        s2[u] = live[u] ? (first ? other : s) : -INFINITY;
        t1 = fmaxf(t1, s1[u]);
        t2 = fmaxf(t2, s2[u]);
      }
      // (a slot that has met no key yet has nothing to scale: the selection, which changes no result, keeps the loop's
      // registers in bounds, 4 x 32,760 keys 141 us with it and 145 without)
      const float g1 = t1 == kDecNone ? 0.f : ex2_approx(m1[i] - t1), g2 = t2 == kDecNone ? 0.f : ex2_approx(m2[i] - t2);
      l1[i] *= g1;
      l2[i] *= g2;
#pragma unroll
      for (int f = 0; f < 8; ++f) acc1[i][f] *= g1, acc2[i][f] *= g2;
#pragma unroll
      for (int u = 0; u < DEEP; ++u) {
        const float p1 = live[u] ? ex2_approx(s1[u] - t1) : 0.f, p2 = live[u] ? ex2_approx(s2[u] - t2) : 0.f;
        float v8[8];
        widen8(vr[u], v8);
        l1[i] += p1;
        l2[i] += p2;
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          acc1[i][f] = fmaf(p1, v8[f], acc1[i][f]);
          acc2[i][f] = fmaf(p2, v8[f], acc2[i][f]);
        }
      }
      m1[i] = t1;
      m2[i] = t2;
    }
  };
  for (int base = k0 + warp * KPW; base < k1; base += 2 * STEP) {  // (the same in all lanes)
    fetch(base + STEP, kr[1], vr[1]);
    work(base, kr[0], vr[0]);
    fetch(base + 2 * STEP, kr[0], vr[0]);
    work(base + STEP, kr[1], vr[1]);
  }
  // the key slots of a warp, then the warps
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
#pragma unroll
    for (int o = LPK; o < 32; o *= 2) {
      float b1[8], b2[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        b1[f] = __shfl_xor_sync(0xffffffffu, acc1[i][f], o);
        b2[f] = __shfl_xor_sync(0xffffffffu, acc2[i][f], o);
      }
      join(m1[i], l1[i], acc1[i], __shfl_xor_sync(0xffffffffu, m1[i], o), __shfl_xor_sync(0xffffffffu, l1[i], o), b1);
      join(m2[i], l2[i], acc2[i], __shfl_xor_sync(0xffffffffu, m2[i], o), __shfl_xor_sync(0xffffffffu, l2[i], o), b2);
    }
    if (slot == 0) {
#pragma unroll
      for (int f = 0; f < 8; f += 4) {
        *reinterpret_cast<float4*>(&sacc[i][0][warp][part * 8 + f]) =
            make_float4(acc1[i][f], acc1[i][f + 1], acc1[i][f + 2], acc1[i][f + 3]);
        *reinterpret_cast<float4*>(&sacc[i][1][warp][part * 8 + f]) =
            make_float4(acc2[i][f], acc2[i][f + 1], acc2[i][f + 2], acc2[i][f + 3]);
      }
    }
    if (lane == 0) sm[i][0][warp] = m1[i], sl[i][0][warp] = l1[i], sm[i][1][warp] = m2[i], sl[i][1][warp] = l2[i];
  }
  __syncthreads();
  // the warps of this CTA: one thread a query, map and feature
  for (int t = threadIdx.x; t < NQ * 2 * D; t += 32 * kDecWarps) {
    const int i = t / (2 * D), x = t / D % 2, f = t % D;
    float m = kDecNone, l = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, sm[i][x][w]);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float g = ex2_approx(sm[i][x][w] - m);
      l += g * sl[i][x][w];
      acc += g * sacc[i][x][w][f];
    }
    cacc[i][x][f] = acc;
    if (f == 0) cm[i][x] = m, cl[i][x] = l;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  // The CTAs of the cluster: CTA c finishes every splits-th value from c on.  All
  // loads of a value are on their way before the first is used.
  const float lam = a.lam_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.lam)[h] << 16)
                               : static_cast<const float*>(a.lam)[h];
  for (int t = split + splits * threadIdx.x; t < NQ * D; t += splits * 32 * kDecWarps) {
    const int i = t / D, f = t % D;
    if (q0 + i >= a.Nq) continue;
    float o[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float pm[kDecSplits], pl[kDecSplits], pa[kDecSplits];
#pragma unroll
      for (int c = 0; c < kDecSplits; ++c) {
        pm[c] = kDecNone, pl[c] = 0.f, pa[c] = 0.f;
        if (c < splits) {
          pm[c] = *cluster.map_shared_rank(&cm[i][x], c);
          pl[c] = *cluster.map_shared_rank(&cl[i][x], c);
          pa[c] = *cluster.map_shared_rank(&cacc[i][x][f], c);
        }
      }
      float m = kDecNone, l = 0.f, acc = 0.f;
#pragma unroll
      for (int c = 0; c < kDecSplits; ++c) m = fmaxf(m, pm[c]);
#pragma unroll
      for (int c = 0; c < kDecSplits; ++c) {
        const float g = ex2_approx(pm[c] - m);
        l += g * pl[c];
        acc += g * pa[c];
      }
      o[x] = acc / l;
    }
    const uint32_t y = len > 0 ? pack_bf16x2(fmaf(-lam, o[1], o[0]), 0.f) : 0u;
    a.out[(((int64_t)b * a.Nq + q0 + i) * a.heads + h) * D + f] = (uint16_t)(y & 0xFFFFu);
  }
  cluster.sync();  // a CTA's shared memory outlives its last reader
}

// Splits of a (b, h)'s keys.  The CTAs fill the machine once, and clusters only
// nine tenths of it: they do not fit into what other clusters leave of a GPC, and a
// second wave costs as much as the first (48 units: 5 splits 138 us, 6 splits 201).
// Where that would leave more than a quarter of the machine idle, many small CTAs
// in several waves (192 units: 1 split 161 us, 4 splits 142).  256 keys a CTA at
// least, 16 CTAs a cluster at most.
template <int NQ>
int decode_splits(int64_t units, int cap) {
  const int64_t once = 134 * DecCfg<NQ>::CTAS / units;
  const int64_t want = once >= 3 ? once : (370 * DecCfg<NQ>::CTAS + units - 1) / units;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, ((int64_t)cap + 255) / 256, kDecSplits}));
}

template <int D, int NQ>
cudaError_t launch_diff_decode_t(const DiffDecodeArgs& a, cudaStream_t s) {
  const int splits = decode_splits<NQ>((int64_t)a.B * a.heads * ((a.Nq + NQ - 1) / NQ), a.cap);
  if (splits > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute(diff_decode_kernel<D, NQ>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * a.heads * splits), (unsigned)((a.Nq + NQ - 1) / NQ));
  cfg.blockDim = dim3(32 * kDecWarps);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)splits;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, diff_decode_kernel<D, NQ>, a, splits);
}

template <int D>
cudaError_t launch_diff_decode_d(const DiffDecodeArgs& a, cudaStream_t s) {
  if (a.Nq == 1) return launch_diff_decode_t<D, 1>(a, s);
  return launch_diff_decode_t<D, 2>(a, s);
}

}  // namespace

cudaError_t launch_diff_decode(const DiffDecodeArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_diff_decode_d<64>(a, s) : launch_diff_decode_d<128>(a, s);
}

}  // namespace salad
