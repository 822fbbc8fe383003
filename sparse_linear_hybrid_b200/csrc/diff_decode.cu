// Differential attention (diff.cu) of a few query rows, one to four in general,
// against a cache of keys and values: query i of sequence b sees keys [0, lens[b])
// (0 keys: the output is 0).
//
// Bound by memory: each live key and value is read once per group of up to four
// queries.  The keys of a (b, h) are split over the CTAs of a cluster (up to 16)
// so that a short batch still fills the machine; every warp keeps an online
// softmax of its keys (running maxima, sums and weighted values of both maps in
// fp32 registers, d/8 lanes a key, eight features a lane), the warps join in
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
constexpr int kDecDeep = 4;  // keys in flight a lane group

// Joins (m, l, acc) of another part into this one.
template <int E>
__device__ __forceinline__ void join(float& m, float& l, float (&acc)[E], float m2, float l2, const float (&acc2)[E]) {
  const float top = fmaxf(m, m2);
  const float a = m == -INFINITY ? 0.f : ex2_approx(m - top), b = m2 == -INFINITY ? 0.f : ex2_approx(m2 - top);
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

template <int D, int NQ>
__global__ void __launch_bounds__(32 * kDecWarps)
    diff_decode_kernel(const DiffDecodeArgs a, int splits) {
  constexpr int LPK = D / 8;          // lanes a key
  constexpr int KPW = 32 / LPK;       // keys a warp takes at once
  // per query and map: maximum, sum, weighted values of the warps, then of the CTA
  __shared__ float sm[NQ][2][kDecWarps], sl[NQ][2][kDecWarps];
  __shared__ __align__(16) float sacc[NQ][2][kDecWarps][D];
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
    m1[i] = m2[i] = -INFINITY;
    l1[i] = l2[i] = 0.f;
#pragma unroll
    for (int f = 0; f < 8; ++f) acc1[i][f] = acc2[i][f] = 0.f;
  }
  const int64_t row = (int64_t)a.heads * D;
  const uint16_t* kp = a.k + (int64_t)b * a.cap * row + (int64_t)h * D + part * 8;
  const uint16_t* vp = a.v + (int64_t)b * a.cap * row + (int64_t)h * D + part * 8;
  const bool first = part < LPK / 2;
  for (int base = k0 + warp * KPW; base < k1; base += kDecWarps * KPW * kDecDeep) {  // (the same in all lanes)
    uint4 kr[kDecDeep], vr[kDecDeep];
    bool live[kDecDeep];
#pragma unroll
    for (int u = 0; u < kDecDeep; ++u) {
      const int key = base + u * kDecWarps * KPW + slot;
      live[u] = key < k1;
      kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
      if (live[u]) {
        kr[u] = __ldcs(reinterpret_cast<const uint4*>(kp + key * row));
        vr[u] = __ldcs(reinterpret_cast<const uint4*>(vp + key * row));
      }
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float s1[kDecDeep], s2[kDecDeep], t1 = m1[i], t2 = m2[i];
#pragma unroll
      for (int u = 0; u < kDecDeep; ++u) {
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
      // (a slot that has met no key yet keeps -inf: its factors are taken as 0)
      const float g1 = t1 == -INFINITY ? 0.f : ex2_approx(m1[i] - t1), g2 = t2 == -INFINITY ? 0.f : ex2_approx(m2[i] - t2);
      l1[i] *= g1;
      l2[i] *= g2;
#pragma unroll
      for (int f = 0; f < 8; ++f) acc1[i][f] *= g1, acc2[i][f] *= g2;
#pragma unroll
      for (int u = 0; u < kDecDeep; ++u) {
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
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  // The warps of every CTA of the cluster, one thread an output feature: CTA c
  // takes the features f with f % splits == c.
  const float lam = a.lam_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.lam)[h] << 16)
                               : static_cast<const float*>(a.lam)[h];
  const int mine = D / splits;  // (splits <= 16 divides d)
  for (int t = threadIdx.x; t < NQ * mine; t += 32 * kDecWarps) {
    const int i = t / mine, f = split * mine + t % mine;
    if (q0 + i >= a.Nq) continue;
    float o[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float m = -INFINITY, l = 0.f, acc[1] = {0.f};
      for (int c = 0; c < splits; ++c) {
        const float* pm = cluster.map_shared_rank(&sm[i][x][0], c);
        const float* pl = cluster.map_shared_rank(&sl[i][x][0], c);
        const float* pa = cluster.map_shared_rank(&sacc[i][x][0][f], c);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float one[1] = {pa[w * D]};
          join(m, l, acc, pm[w], pl[w], one);
        }
      }
      o[x] = len > 0 ? acc[0] / l : 0.f;
    }
    const uint32_t y = pack_bf16x2(fmaf(-lam, o[1], o[0]), 0.f);
    a.out[(((int64_t)b * a.Nq + q0 + i) * a.heads + h) * D + f] = (uint16_t)(y & 0xFFFFu);
  }
  cluster.sync();  // a CTA's shared memory outlives its last reader
}

template <int D, int NQ>
cudaError_t launch_diff_decode_t(const DiffDecodeArgs& a, cudaStream_t s) {
  // Enough CTAs for two an SM, at least 64 keys each, at most 16 in a cluster.
  const int64_t units = (int64_t)a.B * a.heads * ((a.Nq + NQ - 1) / NQ);
  int splits = 1;
  while (splits < 16 && units * splits < 296 && (int64_t)a.cap > 64 * splits) splits *= 2;
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
  if (a.Nq == 2) return launch_diff_decode_t<D, 2>(a, s);
  return launch_diff_decode_t<D, 4>(a, s);
}

}  // namespace

cudaError_t launch_diff_decode(const DiffDecodeArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_diff_decode_d<64>(a, s) : launch_diff_decode_d<128>(a, s);
}

}  // namespace salad
