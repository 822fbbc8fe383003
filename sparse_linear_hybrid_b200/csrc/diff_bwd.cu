// Backward pass of differential attention (diff.cu).  With p_m,ij =
// exp(scale s_m,ij - lse_m,i) over the kept keys, o_2 the second map's output
// and out = o_1 - lam o_2 (both kept by the forward):
//   dp_ij  = dout_i . v_j,   D_2,i = dout_i . o_2,i,   D_1,i = dout_i . out_i + lam D_2,i
//   ds_m   = p_m (dp - D_m)
//   dq_1,i = scale sum_j ds_1,ij k_1,j,  dq_2,i = -lam scale sum_j ds_2,ij k_2,j, dk likewise
//   dv_j   = sum_i (p_1 - lam p_2)_ij dout_i,    dlam = -sum_ij p_2,ij dp_ij
// The maps share dp and dv, so a pair of tiles costs the same products as one
// plain attention head of width d; the exponentials are doubled.
//   diff_prep_kernel  D_1, D_2 and the log-sum-exps in base 2, rows padded to
//                     whole tiles (pad rows: p = 0)
//   diff_dq_kernel    one CTA per (query tile, b, h): S_1, S_2 and dP in tensor
//                     memory, one thread a row and half of the keys; dS_1 and
//                     dS_2 as bf16 over the dP columns that the thread has read;
//                     and the CTA's share of dlam, in fp32 from p and dp themselves
//   diff_dkdv_kernel  one CTA per (key tile, b, h) over the query tiles that keep
//                     it, 64 queries a step: S_1^T, S_2^T, dP^T, then (P_1 - lam
//                     P_2)^T, dS_1^T and dS_2^T as bf16 over the scores' columns
//   diff_dlam_kernel  sums the shares of every head in a fixed order
// Gradients are rounded once, to bf16 (dlam to lam's type).  Warp roles and waits
// as in bwd.cu.
#include "internal.h"
#include "ptx.cuh"

namespace salad {
namespace {

constexpr int kDiffBwdThreads = 320;  // producer/issuer, TMEM owner, eight row warps
constexpr uint64_t kDiffBwdDrainNs = 1000000000ull;
constexpr float kDiffLog2e = 1.4426950408889634f;

struct DiffBwdShared {
  uint64_t fixed_full;
  uint64_t ring_full[2];
  uint64_t k_full[3], v_full[2];
  uint64_t s_full, dp_full, s_read, ds_full, mm_done, grads_done;
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
  float part[8];  // dlam by warp
};

template <int D>
struct DiffBwdCfg {
  static constexpr int DCH = D / 64;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int OFF_FIX = 0;  // two fixed tiles
  // dQ kernel: a three-stage K ring and a two-stage V ring
  static constexpr int DQ_OFF_K = 2 * TILE;
  static constexpr int DQ_OFF_V = 5 * TILE;
  static constexpr int DQ_OFF_BAR = 7 * TILE;
  static constexpr int DQ_USED = DQ_OFF_BAR + (int)sizeof(DiffBwdShared) + 1024;
  static constexpr int DQ_SMEM = DQ_USED > 122880 ? DQ_USED : 122880;
  // dK/dV kernel: two stages of Q, dO and the four row vectors
  static constexpr int VEC = 4 * 128 * 4;
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_VEC = 6 * TILE;
  static constexpr int OFF_BAR = OFF_VEC + 2 * VEC;
  static constexpr int USED = OFF_BAR + (int)sizeof(DiffBwdShared) + 1024;
  static constexpr int SMEM = USED > 122880 ? USED : 122880;
  static constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
  static constexpr uint32_t IDESC_SH = idesc_bf16(128, 64, false, false);  // 64 queries
  static constexpr uint32_t IDESC_H = idesc_bf16(128, 64, false, true);    // gradient of one half of q or k
  static constexpr uint32_t IDESC_V = idesc_bf16(128, D, false, true);
  static_assert(DQ_SMEM <= 232448 && SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void diff_bwd_timeout(DiffBwdShared* sh, uint32_t* status) {
  sh->abort_flag = 1;
  atomicOr(status, kStatusTimeout);
}
__device__ __forceinline__ float diff_lambda(const void* lam, int bf16, int h) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(lam)[h] << 16) : static_cast<const float*>(lam)[h];
}

// K-steps [first, first + count) of X Y^T (both K-major, 128-byte rows in 64-feature chunks of
// `chunk` bytes) into D; the first one overwrites.
template <int COUNT>
__device__ __forceinline__ void mma_steps(uint32_t d_tmem, uint32_t x, uint32_t y, int first, uint32_t idesc) {
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    const int f = first + i;
    const uint32_t off = (f / 4) * 16384 + (f % 4) * 32;
    mma_bf16_ss(d_tmem, sw128_desc(x + off, 16, 1024), sw128_desc(y + off, 16, 1024), idesc, i > 0 ? 1u : 0u);
  }
}

// rows[4][B*Hh][npad]: lse_1 and lse_2 (base 2; +inf in pad rows), D_1, D_2.
// D/8 lanes a row, eight features a lane.
template <int D>
__global__ void __launch_bounds__(256)
    diff_prep_kernel(const uint16_t* __restrict__ out, const uint16_t* __restrict__ out2,
                     const uint16_t* __restrict__ dout, const float* __restrict__ lse, const void* __restrict__ lam,
                     int lam_bf16, int B, int N, int heads, int npad, float* __restrict__ rows) {
  constexpr int LANES = D / 8;
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int64_t total = (int64_t)B * heads * npad;
  const int part = threadIdx.x % LANES;
  if (t >= total) return;  // (whole groups of lanes leave; total is a multiple of 128 rows, so whole CTAs do)
  // rows of neighbouring heads of a token lie side by side: h fastest
  const int h = (int)(t % heads), n = (int)(t / heads % npad), b = (int)(t / heads / npad);
  const int64_t bh = (int64_t)b * heads + h, at = bh * npad + n;
  float d0 = 0.f, d2 = 0.f;
  if (n < N) {
    const int64_t off = (((int64_t)b * N + n) * heads + h) * D + part * 8;
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(out + off)), y = __ldcs(reinterpret_cast<const uint4*>(out2 + off));
    const uint4 g = *reinterpret_cast<const uint4*>(dout + off);
    const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w}, ga[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g0 = bf16_lo_to_f32(ga[i]), g1 = bf16_hi_to_f32(ga[i]);
      d0 = fmaf(bf16_lo_to_f32(xa[i]), g0, fmaf(bf16_hi_to_f32(xa[i]), g1, d0));
      d2 = fmaf(bf16_lo_to_f32(ya[i]), g0, fmaf(bf16_hi_to_f32(ya[i]), g1, d2));
    }
  }
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) {
    d0 += __shfl_xor_sync(0xffffffffu, d0, o);
    d2 += __shfl_xor_sync(0xffffffffu, d2, o);
  }
  if (part == 0) {
    const int64_t BH = (int64_t)B * heads;
    rows[at] = n < N ? lse[bh * N + n] * kDiffLog2e : INFINITY;
    rows[total + at] = n < N ? lse[(BH + bh) * N + n] * kDiffLog2e : INFINITY;
    rows[2 * total + at] = fmaf(diff_lambda(lam, lam_bf16, h), d2, d0);
    rows[3 * total + at] = d2;
  }
}

// p = 2^(s c - l) for 32 scores of a row, 0 from column `valid` on.
__device__ __forceinline__ void diff_exp32(const uint32_t (&sr)[32], float c, float l, int valid, float* p) {
  const uint64_t c2 = f32x2_pack(c, c), nl = f32x2_pack(-l, -l);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x = f32x2_fma(f32x2_pack(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1])), c2, nl);
    float p0, p1;
    if ((i & 3) == 3) {
      exp2_fma_x2(x, p0, p1);
    } else {
      float x0, x1;
      f32x2_unpack(x, x0, x1);
      p0 = ex2_approx(x0);
      p1 = ex2_approx(x1);
    }
    p[2 * i] = 2 * i < valid ? p0 : 0.f;
    p[2 * i + 1] = 2 * i + 1 < valid ? p1 : 0.f;
  }
}

// 32 fp32 columns of tensor memory times mul, as bf16 to 64 bytes of global memory.
__device__ __forceinline__ void store_bf16_32(uint16_t* dst, const uint32_t (&g)[32], float mul) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    *reinterpret_cast<uint4*>(dst + i) =
        make_uint4(pack_bf16x2(__uint_as_float(g[i]) * mul, __uint_as_float(g[i + 1]) * mul),
                   pack_bf16x2(__uint_as_float(g[i + 2]) * mul, __uint_as_float(g[i + 3]) * mul),
                   pack_bf16x2(__uint_as_float(g[i + 4]) * mul, __uint_as_float(g[i + 5]) * mul),
                   pack_bf16x2(__uint_as_float(g[i + 6]) * mul, __uint_as_float(g[i + 7]) * mul));
}

// ------------------------------------------------------------------ dQ
template <int D>
__global__ void __launch_bounds__(kDiffBwdThreads, 1)
    diff_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                   const int32_t* __restrict__ row_ptr, const int32_t* __restrict__ col_idx,
                   const float* __restrict__ rows, const void* __restrict__ lam, int lam_bf16,
                   uint16_t* __restrict__ dq, float* __restrict__ dlam_part, int N, int heads, int nb, int npad,
                   int mask_per_bh, float scale, float scale_log2, uint32_t* status, uint64_t limit_ns) {
  using C = DiffBwdCfg<D>;
  // S_1 [0,128), S_2 [128,256), dP [256,384): a thread's half e of the keys is
  // dP [256 + 64 e, +64), over which it writes dS_1 (32 columns) and dS_2 (32);
  // dQ_1 [384,448), dQ_2 [448,512).  At d = 64 the two products take both halves
  // of k (N = 64) and the half that does not belong is left aside.
  constexpr uint32_t TM_S = 0, TM_DP = 256, TM_DQ = 384;
  extern __shared__ uint8_t diff_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(diff_smem_raw) + 1023) & ~uintptr_t(1023));
  DiffBwdShared* sh = reinterpret_cast<DiffBwdShared*>(smem + C::DQ_OFF_BAR);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qt = blockIdx.x % nb, bh = blockIdx.x / nb, b = bh / heads, h = bh % heads;
  const int mrow = (mask_per_bh ? bh : h) * nb + qt;
  const int mask_rows = (mask_per_bh ? (int)(gridDim.x / nb) : heads) * nb;
  const int c0 = row_ptr[mrow];
  const int n = debug_row_ok(row_ptr, col_idx, mrow, mask_rows, nb, true, status) ? row_ptr[mrow + 1] - c0 : 0;

  if (threadIdx.x == 0) {
    mbar_init(&sh->fixed_full, 1);
    for (int st = 0; st < 3; ++st) mbar_init(&sh->k_full[st], 1);
    for (int st = 0; st < 2; ++st) mbar_init(&sh->v_full[st], 1);
    mbar_init(&sh->dp_full, 1);
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->s_read, 8);
    mbar_init(&sh->ds_full, 8);
    mbar_init(&sh->mm_done, 1);
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const uint32_t q_s = sbase + C::OFF_FIX, do_s = q_s + C::TILE;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int kl = 0, vl = 0;  // K and V loads issued
      auto load_k = [&](int j) {
        const int st = j % 3, col = col_idx[c0 + j];
        mbar_arrive_expect_tx(&sh->k_full[st], C::TILE);
#pragma unroll
        for (int ch = 0; ch < C::DCH; ++ch)
          tma_load_3d(smem + C::DQ_OFF_K + st * C::TILE + ch * 16384, &tm_k, &sh->k_full[st], h * D + ch * 64,
                      col * 128, b);
        ++kl;
      };
      auto load_v = [&](int j) {
        const int st = j & 1, col = col_idx[c0 + j];
        mbar_arrive_expect_tx(&sh->v_full[st], C::TILE);
#pragma unroll
        for (int ch = 0; ch < C::DCH; ++ch)
          tma_load_3d(smem + C::DQ_OFF_V + st * C::TILE + ch * 16384, &tm_v, &sh->v_full[st], h * D + ch * 64,
                      col * 128, b);
        ++vl;
      };
      auto k_tile = [&](int j) { return sbase + C::DQ_OFF_K + (j % 3) * C::TILE; };
      auto v_tile = [&](int j) { return sbase + C::DQ_OFF_V + (j & 1) * C::TILE; };
      auto wait_k = [&](int j) { return mbar_wait(&sh->k_full[j % 3], (uint32_t)((j / 3) & 1), limit_ns); };
      auto wait_v = [&](int j) { return mbar_wait(&sh->v_full[j & 1], (uint32_t)((j >> 1) & 1), limit_ns); };
      auto issue_s = [&](int j) {
        mma_steps<D / 32>(tmem + TM_S, q_s, k_tile(j), 0, C::IDESC_S);
        mma_steps<D / 32>(tmem + TM_S + 128, q_s, k_tile(j), D / 32, C::IDESC_S);
        mma_commit(&sh->s_full);
      };
      auto issue_dp = [&](int j) {
        mma_steps<D / 16>(tmem + TM_DP, do_s, v_tile(j), 0, C::IDESC_S);
        mma_commit(&sh->dp_full);
      };
      mbar_arrive_expect_tx(&sh->fixed_full, 2 * C::TILE);
#pragma unroll
      for (int ch = 0; ch < C::DCH; ++ch) {
        tma_load_3d(smem + C::OFF_FIX + ch * 16384, &tm_q, &sh->fixed_full, h * D + ch * 64, qt * 128, b);
        tma_load_3d(smem + C::OFF_FIX + C::TILE + ch * 16384, &tm_do, &sh->fixed_full, h * D + ch * 64, qt * 128, b);
      }
      for (int j = 0; j < n && j < 3; ++j) load_k(j);
      for (int j = 0; j < n && j < 2; ++j) load_v(j);
      // S of the next tile as soon as the row warps hold S in registers; then the
      // gradient products and, behind them in the issue order, dP of the next
      // tile over dS.  K_{j+3} refills K_j's stage once the gradient products
      // have read it, V_{j+2} V_j's once dP_j is done.
      ok = mbar_wait(&sh->fixed_full, 0, limit_ns);
      if (ok && n >= 1) {
        ok = wait_k(0) && wait_v(0);
        if (ok) {
          tc_fence_after();
          issue_s(0);
          issue_dp(0);
        }
      }
      for (int j = 0; ok && j < n; ++j) {
        if (j + 1 < n) {
          if (sh->abort_flag || !mbar_wait(&sh->s_read, (uint32_t)(j & 1), limit_ns) || !wait_k(j + 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue_s(j + 1);
        }
        if (sh->abort_flag || !mbar_wait(&sh->ds_full, (uint32_t)(j & 1), limit_ns)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(tmem + TM_DQ + 64 * m, tmem + TM_DP + 64 * (kk >> 2) + 32 * m + 8 * (kk & 3),
                        sw128_desc(k_tile(j) + (C::DCH == 2 ? m * 16384 : 0) + kk * 2048, 16384, 1024), C::IDESC_H,
                        (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&sh->mm_done);
        // dP_j completed before the row warps formed dS_j: V_j's stage is free
        if (j + 2 < n) load_v(j + 2);
        if (j + 1 < n) {
          if (!wait_v(j + 1)) { ok = false; break; }
          tc_fence_after();
          issue_dp(j + 1);
        }
        if (j + 3 < n) {
          if (!mbar_wait(&sh->mm_done, (uint32_t)(j & 1), limit_ns)) { ok = false; break; }
          load_k(j + 3);
        }
      }
      if (!ok) diff_bwd_timeout(sh, status);
      // every product has ended before the tensor memory is given back, also when a row warp gave up
      mma_commit(&sh->drain);
      mbar_wait(&sh->drain, 0, kDiffBwdDrainNs);
      // every copy this thread started lands before the CTA exits
      mbar_wait(&sh->fixed_full, 0, kDiffBwdDrainNs);
      for (int i = (kl > 3 ? kl - 3 : 0); i < kl; ++i)
        mbar_wait(&sh->k_full[i % 3], (uint32_t)((i / 3) & 1), kDiffBwdDrainNs);
      for (int i = (vl > 2 ? vl - 2 : 0); i < vl; ++i)
        mbar_wait(&sh->v_full[i & 1], (uint32_t)((i >> 1) & 1), kDiffBwdDrainNs);
    }
  } else if (warp >= 2) {
    // one thread a query row and half of the keys of every tile
    const int quarter = warp & 3, r = quarter * 32 + lane, half = (warp - 2) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    const size_t total = (size_t)(gridDim.x / nb) * npad, at = (size_t)bh * npad + qt * 128 + r;
    const float l1 = rows[at], l2 = rows[total + at], D1 = rows[2 * total + at], D2 = rows[3 * total + at];
    float dl = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int valid = N - col_idx[c0 + j] * 128 - 64 * half;  // real keys from this half's first on
      if (!mbar_wait_warp(&sh->s_full, (uint32_t)(j & 1), limit_ns)) { ok = false; break; }
      tc_fence_after();
      float p1[64], p2[64];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t s1[32], s2[32];
        tmem_ld32(lane_addr + TM_S + 64 * half + 32 * c, s1);
        tmem_ld32(lane_addr + TM_S + 128 + 64 * half + 32 * c, s2);
        tmem_ld_wait();
        diff_exp32(s1, scale_log2, l1, valid - 32 * c, p1 + 32 * c);
        diff_exp32(s2, scale_log2, l2, valid - 32 * c, p2 + 32 * c);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->s_read);
      if (!mbar_wait_warp(&sh->dp_full, (uint32_t)(j & 1), limit_ns)) { ok = false; break; }
      tc_fence_after();
      {
        uint32_t pr[2][32];
        tmem_ld32(lane_addr + TM_DP + 64 * half, pr[0]);
        tmem_ld32(lane_addr + TM_DP + 64 * half + 32, pr[1]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t a[16], z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int e = 32 * c + 2 * i;
            const float g0 = __uint_as_float(pr[c][2 * i]), g1 = __uint_as_float(pr[c][2 * i + 1]);
            a[i] = pack_bf16x2(p1[e] * (g0 - D1), p1[e + 1] * (g1 - D1));
            z[i] = pack_bf16x2(p2[e] * (g0 - D2), p2[e + 1] * (g1 - D2));
            dl = fmaf(p2[e], g0, fmaf(p2[e + 1], g1, dl));
          }
          tmem_st16(lane_addr + TM_DP + 64 * half + 16 * c, a);
          tmem_st16(lane_addr + TM_DP + 64 * half + 32 + 16 * c, z);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->ds_full);
    }
    if (ok && n >= 1) ok = mbar_wait_warp(&sh->mm_done, (uint32_t)((n - 1) & 1), limit_ns);
    if (!ok) {
      diff_bwd_timeout(sh, status);
    } else {
      tc_fence_after();
      const int row = qt * 128 + r;
      const float mul = half ? -diff_lambda(lam, lam_bf16, h) * scale : scale;  // half: the map whose dq this thread writes
      uint16_t* dst = dq + (((size_t)b * N + row) * heads + h) * D + half * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t g[32];
        if (n >= 1) {
          tmem_ld32(lane_addr + TM_DQ + 64 * half + (D == 64 ? 32 * half : 32 * c), g);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = 0u;
        }
        if (row < N) store_bf16_32(dst + 32 * c, g, n >= 1 ? mul : 0.f);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) dl += __shfl_xor_sync(0xffffffffu, dl, o);
    if (lane == 0) sh->part[warp - 2] = dl;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int i = 0; i < 8; ++i) s += sh->part[i];
    dlam_part[blockIdx.x] = s;
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dK, dV
template <int D>
__global__ void __launch_bounds__(kDiffBwdThreads, 1)
    diff_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const int32_t* __restrict__ t_row_ptr, const int32_t* __restrict__ t_col_idx,
                     const float* __restrict__ rows, const void* __restrict__ lam, int lam_bf16,
                     uint16_t* __restrict__ dk, uint16_t* __restrict__ dv, int N, int heads, int nb, int npad,
                     int mask_per_bh, float scale, float scale_log2, uint32_t* status, uint64_t limit_ns) {
  using C = DiffBwdCfg<D>;
  // 64 queries a step.  S_1^T [0,64), S_2^T [64,128), dP^T [128,192); a thread's
  // half e of the queries is columns [32 e, +32) of each, and it writes (P_1 - lam
  // P_2)^T at [32 e, +16), dS_1^T at [32 e + 16, +16) and dS_2^T at [64 + 32 e, +16).
  // dV [192,192+d), dK_1 [320,384), dK_2 [384,448) (at d = 64 both halves of q,
  // as in the dQ kernel).
  constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 192, TM_DK = 320;
  extern __shared__ uint8_t diff_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(diff_smem_raw) + 1023) & ~uintptr_t(1023));
  DiffBwdShared* sh = reinterpret_cast<DiffBwdShared*>(smem + C::OFF_BAR);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kt = blockIdx.x % nb, bh = blockIdx.x / nb, b = bh / heads, h = bh % heads;
  const int mrow = (mask_per_bh ? bh : h) * nb + kt;
  const int mask_rows = (mask_per_bh ? (int)(gridDim.x / nb) : heads) * nb;
  const int c0 = t_row_ptr[mrow];
  const int n =
      debug_row_ok(t_row_ptr, t_col_idx, mrow, mask_rows, nb, true, status) ? t_row_ptr[mrow + 1] - c0 : 0;

  if (threadIdx.x == 0) {
    mbar_init(&sh->fixed_full, 1);
    mbar_init(&sh->ring_full[0], 1);
    mbar_init(&sh->ring_full[1], 1);
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->ds_full, 8);
    mbar_init(&sh->grads_done, 1);
    mbar_init(&sh->mm_done, 1);
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const uint32_t k_s = sbase + C::OFF_FIX, v_s = k_s + C::TILE;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int loads = 0;
      auto load_q = [&](int j) {
        const int s = j & 1, qi = t_col_idx[c0 + j];
        uint8_t* dst = smem + C::OFF_RING + s * 2 * C::TILE;
        float* vec = reinterpret_cast<float*>(smem + C::OFF_VEC + s * C::VEC);
        mbar_arrive_expect_tx(&sh->ring_full[s], 2 * C::TILE + C::VEC);
#pragma unroll
        for (int ch = 0; ch < C::DCH; ++ch) {
          tma_load_3d(dst + ch * 16384, &tm_q, &sh->ring_full[s], h * D + ch * 64, qi * 128, b);
          tma_load_3d(dst + C::TILE + ch * 16384, &tm_do, &sh->ring_full[s], h * D + ch * 64, qi * 128, b);
        }
        const size_t total = (size_t)(gridDim.x / nb) * npad, at = (size_t)bh * npad + (size_t)qi * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) bulk_load(vec + 128 * i, rows + i * total + at, 512, &sh->ring_full[s]);
        ++loads;
      };
      // scores and dP^T of step i (64 queries of tile i / 2)
      auto issue_s = [&](int i) {
        const uint32_t qs = sbase + C::OFF_RING + ((i >> 1) & 1) * 2 * C::TILE + (i & 1) * 8192;
        mma_steps<D / 32>(tmem + TM_S, k_s, qs, 0, C::IDESC_SH);
        mma_steps<D / 32>(tmem + TM_S + 64, k_s, qs, D / 32, C::IDESC_SH);
        mma_steps<D / 16>(tmem + TM_DP, v_s, qs + C::TILE, 0, C::IDESC_SH);
        mma_commit(&sh->s_full);
      };
      mbar_arrive_expect_tx(&sh->fixed_full, 2 * C::TILE);
#pragma unroll
      for (int ch = 0; ch < C::DCH; ++ch) {
        tma_load_3d(smem + C::OFF_FIX + ch * 16384, &tm_k, &sh->fixed_full, h * D + ch * 64, kt * 128, b);
        tma_load_3d(smem + C::OFF_FIX + C::TILE + ch * 16384, &tm_v, &sh->fixed_full, h * D + ch * 64, kt * 128, b);
      }
      for (int j = 0; j < n && j < 2; ++j) load_q(j);
      ok = mbar_wait(&sh->fixed_full, 0, limit_ns);
      if (ok && n >= 1) {
        ok = mbar_wait(&sh->ring_full[0], 0, limit_ns);
        if (ok) {
          tc_fence_after();
          issue_s(0);
        }
      }
      for (int i = 0; ok && i < 2 * n; ++i) {
        const int j = i >> 1, ph = i & 1;
        const uint32_t qs = sbase + C::OFF_RING + (j & 1) * 2 * C::TILE + ph * 8192;
        if (sh->abort_flag || !mbar_wait(&sh->ds_full, (uint32_t)(i & 1), limit_ns)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t a = tmem + TM_S + 32 * (kk >> 1) + 8 * (kk & 1), acc = (i > 0 || kk > 0) ? 1u : 0u;
          mma_bf16_ts(tmem + TM_DV, a, sw128_desc(qs + C::TILE + kk * 2048, 16384, 1024), C::IDESC_V, acc);
          mma_bf16_ts(tmem + TM_DK, a + 16, sw128_desc(qs + kk * 2048, 16384, 1024), C::IDESC_H, acc);
          mma_bf16_ts(tmem + TM_DK + 64, a + 64, sw128_desc(qs + (C::DCH == 2 ? 16384 : 0) + kk * 2048, 16384, 1024),
                      C::IDESC_H, acc);
        }
        if (i + 1 == 2 * n) {
          mma_commit(&sh->grads_done);
          break;
        }
        if (ph == 1) {
          mma_commit(&sh->mm_done);
          if (!mbar_wait(&sh->ring_full[(j + 1) & 1], (uint32_t)(((j + 1) >> 1) & 1), limit_ns)) { ok = false; break; }
          tc_fence_after();
        }
        issue_s(i + 1);  // over the operands of the products before it, which run first
        if (ph == 1 && j + 2 < n) {
          // the stage of tile j is free once its gradient products have read it
          if (!mbar_wait(&sh->mm_done, (uint32_t)(j & 1), limit_ns)) { ok = false; break; }
          load_q(j + 2);
        }
      }
      if (!ok) diff_bwd_timeout(sh, status);
      // every product has ended before the tensor memory is given back, also when a row warp gave up
      mma_commit(&sh->drain);
      mbar_wait(&sh->drain, 0, kDiffBwdDrainNs);
      mbar_wait(&sh->fixed_full, 0, kDiffBwdDrainNs);
      for (int i = (loads > 2 ? loads - 2 : 0); i < loads; ++i)
        mbar_wait(&sh->ring_full[i & 1], (uint32_t)((i >> 1) & 1), kDiffBwdDrainNs);
    }
  } else if (warp >= 2) {
    // one thread a key row and half of a step's queries
    const int quarter = warp & 3, r = quarter * 32 + lane, half = (warp - 2) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    const float lh = diff_lambda(lam, lam_bf16, h);
    bool ok = true;
    for (int i = 0; i < 2 * n; ++i) {
      const int j = i >> 1, s = j & 1;
      if (!mbar_wait_warp(&sh->s_full, (uint32_t)(i & 1), limit_ns) ||
          !mbar_wait_warp(&sh->ring_full[s], (uint32_t)((j >> 1) & 1), limit_ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float* vec = reinterpret_cast<const float*>(smem + C::OFF_VEC + s * C::VEC) + 64 * (i & 1) + 32 * half;
      uint32_t s1[32], s2[32], pr[32];
      tmem_ld32(lane_addr + TM_S + 32 * half, s1);
      tmem_ld32(lane_addr + TM_S + 64 + 32 * half, s2);
      tmem_ld32(lane_addr + TM_DP + 32 * half, pr);
      tmem_ld_wait();
      uint32_t a[16], z1[16], z2[16];
      const uint64_t c2 = f32x2_pack(scale_log2, scale_log2);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 la = *reinterpret_cast<const float2*>(vec + 2 * k), lb = *reinterpret_cast<const float2*>(vec + 128 + 2 * k);
        const float2 da = *reinterpret_cast<const float2*>(vec + 256 + 2 * k), db = *reinterpret_cast<const float2*>(vec + 384 + 2 * k);
        const uint64_t x1 = f32x2_fma(f32x2_pack(__uint_as_float(s1[2 * k]), __uint_as_float(s1[2 * k + 1])), c2, f32x2_pack(-la.x, -la.y));
        const uint64_t x2 = f32x2_fma(f32x2_pack(__uint_as_float(s2[2 * k]), __uint_as_float(s2[2 * k + 1])), c2, f32x2_pack(-lb.x, -lb.y));
        float p0, p1, q0, q1;
        if ((k & 3) == 3) {
          exp2_fma_x2(x1, p0, p1);
          exp2_fma_x2(x2, q0, q1);
        } else {
          float y0, y1;
          f32x2_unpack(x1, y0, y1);
          p0 = ex2_approx(y0);
          p1 = ex2_approx(y1);
          f32x2_unpack(x2, y0, y1);
          q0 = ex2_approx(y0);
          q1 = ex2_approx(y1);
        }
        const float g0 = __uint_as_float(pr[2 * k]), g1 = __uint_as_float(pr[2 * k + 1]);
        a[k] = pack_bf16x2(fmaf(-lh, q0, p0), fmaf(-lh, q1, p1));
        z1[k] = pack_bf16x2(p0 * (g0 - da.x), p1 * (g1 - da.y));
        z2[k] = pack_bf16x2(q0 * (g0 - db.x), q1 * (g1 - db.y));
      }
      tmem_st16(lane_addr + TM_S + 32 * half, a);
      tmem_st16(lane_addr + TM_S + 32 * half + 16, z1);
      tmem_st16(lane_addr + TM_S + 64 + 32 * half, z2);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->ds_full);
    }
    if (ok && n >= 1) ok = mbar_wait_warp(&sh->grads_done, 0, limit_ns);
    if (!ok) {
      diff_bwd_timeout(sh, status);
    } else {
      tc_fence_after();
      const int row = kt * 128 + r;
      const size_t off = (((size_t)b * N + row) * heads + h) * D + half * (D / 2);
      const float mul = half ? -lh * scale : scale;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t g[32], v[32];
        if (n >= 1) {
          tmem_ld32(lane_addr + TM_DK + 64 * half + (D == 64 ? 32 * half : 32 * c), g);
          tmem_ld32(lane_addr + TM_DV + half * (D / 2) + 32 * c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = v[i] = 0u;
        }
        if (row < N) {
          store_bf16_32(dk + off + 32 * c, g, n >= 1 ? mul : 0.f);
          store_bf16_32(dv + off + 32 * c, v, 1.f);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dlam[h] = -(the shares of every (b, query tile) of the head), one CTA a head, in a fixed order.
__global__ void __launch_bounds__(256)
    diff_dlam_kernel(const float* __restrict__ part, int B, int heads, int nb, void* __restrict__ dlam, int bf16) {
  __shared__ double sum[256];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < (int64_t)B * nb; i += 256)
    s += (double)part[((i / nb) * heads + h) * nb + i % nb];
  sum[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o /= 2) {
    if (threadIdx.x < o) sum[threadIdx.x] += sum[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float v = (float)-sum[0];
    if (bf16)
      static_cast<uint16_t*>(dlam)[h] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
    else
      static_cast<float*>(dlam)[h] = v;
  }
}

template <int D>
cudaError_t launch_diff_bwd_t(const DiffArgs& a, cudaStream_t s) {
  using C = DiffBwdCfg<D>;
  const int64_t lanes = (int64_t)a.B * a.heads * a.npad * (D / 8);
  diff_prep_kernel<D><<<(unsigned)((lanes + 255) / 256), 256, 0, s>>>(a.out, a.out2, a.dout, a.lse, a.lam, a.lam_bf16,
                                                                     a.B, a.N, a.heads, a.npad, a.rows);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int grid = a.B * a.heads * a.nb;
  e = cudaFuncSetAttribute(diff_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::DQ_SMEM);
  if (e != cudaSuccess) return e;
  diff_dq_kernel<D><<<grid, kDiffBwdThreads, C::DQ_SMEM, s>>>(
      *a.tm_q, *a.tm_k, *a.tm_v, *a.tm_do, a.row_ptr, a.col_idx, a.rows, a.lam, a.lam_bf16, a.dq, a.dlam_part, a.N,
      a.heads, a.nb, a.npad, a.mask_per_bh, a.scale, a.scale_log2, a.status, a.wait_limit_ns);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(diff_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  diff_dkdv_kernel<D><<<grid, kDiffBwdThreads, C::SMEM, s>>>(
      *a.tm_q, *a.tm_k, *a.tm_v, *a.tm_do, a.t_row_ptr, a.t_col_idx, a.rows, a.lam, a.lam_bf16, a.dk, a.dv, a.N,
      a.heads, a.nb, a.npad, a.mask_per_bh, a.scale, a.scale_log2, a.status, a.wait_limit_ns);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  diff_dlam_kernel<<<a.heads, 256, 0, s>>>(a.dlam_part, a.B, a.heads, a.nb, a.dlam, a.lam_bf16);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_backward(const DiffArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_diff_bwd_t<64>(a, s) : launch_diff_bwd_t<128>(a, s);
}

}  // namespace salad
