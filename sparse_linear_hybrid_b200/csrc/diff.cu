// Differential attention over the kept key blocks: each head's q and k (d wide)
// hold two halves of h = d/2 features, each half has its own softmax map over
// the same keys, and the maps' difference weighs the values:
//   P_m = softmax(scale Q_m K_m^T) over the kept keys (m = 1, 2)
//   out = P_1 V - lam[head] P_2 V          (0 for a query whose blocks keep no key)
// One CTA takes one 128-row query tile of one (b, h) and walks its kept key
// tiles; both maps read the same K and V tiles.
//
// Tensor memory (512 columns): O_1 [256,256+d), O_2 [384,384+d), and for map m two
// score buffers of 64 keys, [128 m, +64) and [128 m + 64, +64).  A step is 64 keys:
// P_m as bf16 takes the place of the step's scores, and the scores two steps on
// follow P_m V in the issue order, so a map's softmax warps work on one buffer
// while the tensor cores work on the other.  (Score products of 64 keys run at 48
// cycles, not 32: their operands come from shared memory at 128 bytes a cycle.)
// Warp roles, 384 threads: warp 0 TMA producer (K and V rings of three tiles),
// warps 1 and 2 tcgen05 issuers of map 1 and 2 (warp 1 owns the tensor memory),
// warps 4-7 softmax of map 1 and warps 8-11 of map 2, one thread a query row.  Two
// issuers, because issuing slows the other warps of its scheduler.  At the end the
// two warp groups exchange the row sums and each writes half of the features of its
// row.
// Roundings that are choices: P enters its product as bf16 (half a step, 2^-8 of
// each weight at most, as much as the output's own rounding), and the sum that O is
// divided by adds the same rounded p: a weight that holds its row is exact.  The
// log-sum-exp adds the unrounded p.
//
// Bound by the exponentials and their row work.  A step has 900 cycles of products
// (384 scores, 512 P V, at d = 128) and 768 of the special-function unit, with one
// pair of exponentials in four on the FMA pipe (exp2_fma_x2; 32,760 tokens x 12
// heads of 128 at 90 % block sparsity, taken in turn: none 983 us, one in eight 932,
// one in four and three in eight 914, one in two 924), and takes 1,570 (1.68 M active
// cycles an SM over 1,068 steps, the ends of a CTA included; the row warps issue in
// 52 % of the cycles).  Two things that a right row needs are in that: the watch over
// the cubic's range (softmax_pass; 927 -> 935 us taken in turn) and the sum of the
// rounded weights (987 -> 1,032).  In a long run, 1,115 us (0.99 TFLOP of products:
// 890 TFLOP/s).  Every barrier wait is bounded; on a time-out the kernel records it and
// drains.
#include "diff.cuh"
#include "internal.h"

namespace salad {
namespace {

constexpr int kDiffThreads = 384;
constexpr uint64_t kDiffDrainNs = 1000000000ull;
// What a weight and a step's sum of weights may grow to.  O = sum p v has to stay in
// fp32's range: with 2^15 steps (2 million keys) it does for values up to 2^88.
constexpr float kDiffGrownLog2 = 24.f;
constexpr float kDiffGrown = 16777216.f;  // 2^24
constexpr float kLn2 = 0.69314718055994531f;

struct DiffShared {
  uint64_t q_full;
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full[2][2];  // per map and buffer: the scores of a step are in tensor memory
  uint64_t p_full[2][2];  // per map and buffer: the four softmax warps have written P of a step (they may be a step ahead)
  uint64_t pv_done[2];    // per map: P V of a step is done
  uint64_t o_full;      // every product is done
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
  float sum[2][128];    // per map: row sums, for the other group's features
};

template <int D>
struct DiffCfg {
  static constexpr int DCH = D / 64;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int STAGES = 3;
  static constexpr int OFF_Q = 0;                       // later the staged output
  static constexpr int OFF_K = TILE;                    // stage 0 later holds the staged second output
  static constexpr int OFF_V = OFF_K + STAGES * TILE;
  static constexpr int OFF_BAR = OFF_V + STAGES * TILE;
  static constexpr int SMEM_USED = OFF_BAR + (int)sizeof(DiffShared) + 1024;
  // at least 120 KB so that one CTA (and its 512 TMEM columns) owns the SM
  static constexpr int SMEM = SMEM_USED > 122880 ? SMEM_USED : 122880;
  static constexpr uint32_t TM_S = 0, TM_O = 256;       // + 128 per map
  static constexpr uint32_t IDESC_S = idesc_bf16(128, 64, false, false);  // 64 keys
  static constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true);
  static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void diff_timeout(DiffShared* sh, uint32_t* status) {
  sh->abort_flag = 1;
  atomicOr(status, kStatusTimeout);
}

// -inf in place of the scores from column `valid` on.
__device__ __forceinline__ void mask_keys(uint32_t (&sr)[32], int valid) {
  if (valid < 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= valid) sr[i] = __float_as_uint(-INFINITY);
  }
}

__device__ __forceinline__ void max_of(const uint32_t (&sr)[32], float (&m)[4]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = fmax3(m[k], __uint_as_float(sr[i + 2 * k]), __uint_as_float(sr[i + 2 * k + 1]));
}

// The maximum of 64 scores of the row.
__device__ __forceinline__ float row_max(uint32_t s_addr, int valid) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  uint32_t sr[2][32];
  tmem_ld32(s_addr, sr[0]);
  tmem_ld32(s_addr + 32, sr[1]);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    mask_keys(sr[c], valid - 32 * c);
    max_of(sr[c], m);
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// p = 2^(s c + b) of 64 scores of the row as bf16 pairs; returns the sum of those, and
// with TRAIN in `exact` the sum before the rounding.  The cubic wraps around for
// exponents from 128 on (to NaN, negative or small values, which no sum shows) and
// takes NaN for a large negative one, so `top` is the largest exponent that it was
// given, NaN when one of them is.
template <bool TRAIN>
__device__ __forceinline__ float softmax_pass(uint32_t s_addr, int valid, uint64_t c2, float b, uint32_t (&pk)[32],
                                              float& top, float& exact) {
  const uint64_t b2 = f32x2_pack(b, b);
  uint64_t acc0 = 0, acc1 = 0, full = 0;
  top = -INFINITY;
  uint32_t sr[2][32];
  tmem_ld32(s_addr, sr[0]);
  tmem_ld32(s_addr + 32, sr[1]);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t(&x)[32] = sr[c];
    mask_keys(x, valid - 32 * c);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint64_t e = f32x2_fma(f32x2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, b2);
      float p0, p1, x0, x1;
      f32x2_unpack(e, x0, x1);
      if ((i & 3) == 3) {
        exp2_fma_x2(e, p0, p1);
        top = fmax3_nan(top, x0, x1);
      } else {
        p0 = ex2_approx(x0);
        p1 = ex2_approx(x1);
      }
      const uint32_t w = pack_bf16x2(p0, p1);
      pk[16 * c + i] = w;
      if (i & 1)
        acc1 = f32x2_add(acc1, f32x2_pack(bf16_lo_to_f32(w), bf16_hi_to_f32(w)));
      else
        acc0 = f32x2_add(acc0, f32x2_pack(bf16_lo_to_f32(w), bf16_hi_to_f32(w)));
      if (TRAIN) full = f32x2_add(full, f32x2_pack(p0, p1));
    }
  }
  float a0, a1;
  f32x2_unpack(full, a0, a1);
  exact = a0 + a1;
  f32x2_unpack(f32x2_add(acc0, acc1), a0, a1);
  return a0 + a1;
}

// TRAIN: also O_2 / l_2 and the log-sum-exps of both maps.
template <int D, bool TRAIN>
__global__ void __launch_bounds__(kDiffThreads, 1)
    diff_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_out,
                    const __grid_constant__ CUtensorMap tm_out2, const int32_t* __restrict__ row_ptr,
                    const int32_t* __restrict__ col_idx, const void* __restrict__ lam, int lam_bf16,
                    float* __restrict__ lse, int N, int heads, int nb, int mask_per_bh, float scale_log2,
                    uint32_t* status, uint64_t limit_ns) {
  using C = DiffCfg<D>;
  extern __shared__ uint8_t diff_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(diff_smem_raw) + 1023) & ~uintptr_t(1023));
  DiffShared* sh = reinterpret_cast<DiffShared*>(smem + C::OFF_BAR);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t polls = polls_of(limit_ns);
  const int warp = warp_uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int qt = blockIdx.x % nb, bh = blockIdx.x / nb, b = bh / heads, h = bh % heads;
  const int mrow = (mask_per_bh ? bh : h) * nb + qt;
  const int mask_rows = (mask_per_bh ? (int)(gridDim.x / nb) : heads) * nb;
  const int c0 = warp_uniform(row_ptr[mrow]);
  const int n = warp_uniform(debug_row_ok(row_ptr, col_idx, mrow, mask_rows, nb, true, status) ? row_ptr[mrow + 1] - c0 : 0);

  // steps of 64 keys; columns ascend, so only the last tile can be short
  const int last = warp_uniform(n > 0 ? min(128, N - col_idx[c0 + n - 1] * 128) : 0);
  const int steps = 2 * n - (n > 0 && last <= 64 ? 1 : 0);

  if (threadIdx.x == 0) {
    mbar_init(&sh->q_full, 1);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sh->k_full[s], 1);
      mbar_init(&sh->k_empty[s], 2);  // both maps' products
      mbar_init(&sh->v_full[s], 1);
      mbar_init(&sh->v_empty[s], 2);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&sh->s_full[m][0], 1);
      mbar_init(&sh->s_full[m][1], 1);
      mbar_init(&sh->pv_done[m], 1);
      mbar_init(&sh->p_full[m][0], 4);
      mbar_init(&sh->p_full[m][1], 4);
    }
    mbar_init(&sh->o_full, 2);
    mbar_init(&sh->drain, 2);
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
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's: they begin at 0

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
      bool ok = true;
      int kl = 0, vl = 0;
      mbar_arrive_expect_tx(&sh->q_full, C::TILE);
      tma_load_4d(smem + C::OFF_Q, &tm_q, &sh->q_full, 0, qt * 128, h * C::DCH, b);
      for (int j = 0; j < n; ++j) {
        const int s = j % C::STAGES, col = col_idx[c0 + j];
        const uint32_t ph = (uint32_t)((j / C::STAGES) & 1);
        if (!mbar_await_one(&sh->k_empty[s], ph ^ 1, limit_ns)) { ok = false; break; }
        mbar_arrive_expect_tx(&sh->k_full[s], C::TILE);
        tma_load_4d(smem + C::OFF_K + s * C::TILE, &tm_k, &sh->k_full[s], 0, col * 128, h * C::DCH, b);
        ++kl;
        if (!mbar_await_one(&sh->v_empty[s], ph ^ 1, limit_ns)) { ok = false; break; }
        mbar_arrive_expect_tx(&sh->v_full[s], C::TILE);
        tma_load_4d(smem + C::OFF_V + s * C::TILE, &tm_v, &sh->v_full[s], 0, col * 128, h * C::DCH, b);
        ++vl;
      }
      if (!ok) diff_timeout(sh, status);
      // every copy this thread started lands before the CTA exits
      mbar_wait(&sh->q_full, 0, kDiffDrainNs);
      for (int i = (kl > C::STAGES ? kl - C::STAGES : 0); i < kl; ++i)
        mbar_wait(&sh->k_full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), kDiffDrainNs);
      for (int i = (vl > C::STAGES ? vl - C::STAGES : 0); i < vl; ++i)
        mbar_wait(&sh->v_full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), kDiffDrainNs);
    }
  } else if (warp <= 2) {
    // ---------------------------------------------------------- tcgen05 issuer of map m
    if (n > 0) {  // (the whole warp; one lane issues)
      const int m = warp - 1;
      const uint32_t s_t = tmem + C::TM_S + 128 * m, o_t = tmem + C::TM_O + 128 * m;
      // the map's half of the features: chunk m of 64 at d = 128, bytes [64 m, +64) of a row at d = 64
      const uint32_t half = (D == 128 ? 16384u : 64u) * m;
      const uint32_t q_s = sbase + C::OFF_Q + half, k_s = sbase + C::OFF_K + half;
      // scores of step u: keys [64 (u & 1), +64) of the tile in stage s
      auto issue_s = [&](int u, int s) {
        const uint32_t kt = k_s + s * C::TILE + (u & 1) * 8192;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_bf16_ss(s_t + 64 * (u & 1), sw128_desc(q_s + 32 * kk, 16, 1024), sw128_desc(kt + 32 * kk, 16, 1024),
                      C::IDESC_S, kk > 0 ? 1u : 0u);
        mma_commit(&sh->s_full[m][u & 1]);
      };
      bool ok = limit_ns != 0;
      mbar_await(&sh->q_full, 0, polls, ok);
      mbar_await(&sh->k_full[0], 0, polls, ok);
      tc_fence_after();
      if (elect_one() && ok) {
        issue_s(0, 0);
        if (steps > 1) issue_s(1, 0);
        mma_commit(&sh->k_empty[0]);
      }
      int s = 0;
      uint32_t ph = 0;  // stage and parity of the step's tile
      for (int u = 0; u < steps; ++u) {
        const int s1 = s + 1 == C::STAGES ? 0 : s + 1;
        const uint32_t ph1 = s1 == 0 ? ph ^ 1 : ph;
        const bool next = u + 2 < steps;  // the step that takes this one's buffer
        if ((u & 1) == 0) {
          mbar_await(&sh->v_full[s], ph, polls, ok);
          if (next) mbar_await(&sh->k_full[s1], ph1, polls, ok);
        }
        mbar_await(&sh->p_full[m][u & 1], (uint32_t)((u >> 1) & 1), polls, ok);
        tc_fence_after();
        if (elect_one() && ok) {
          const uint32_t vt = sbase + C::OFF_V + s * C::TILE + (u & 1) * 8192;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(o_t, s_t + 64 * (u & 1) + kk * 8, sw128_desc(vt + kk * 2048, 16384, 1024), C::IDESC_PV,
                        (u > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&sh->pv_done[m]);
          if ((u & 1) == 1 || u + 1 == steps) mma_commit(&sh->v_empty[s]);
          if (next) {
            issue_s(u + 2, s1);  // over P, behind the product that reads it
            if ((u & 1) == 1 || u + 3 == steps) mma_commit(&sh->k_empty[s1]);
          }
        }
        if (u & 1) {
          s = s1;
          ph = ph1;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (elect_one() && ok) mma_commit(&sh->o_full);
      if (!ok) diff_timeout(sh, status);
      __syncwarp();
      // every product has ended before the tensor memory is given back, also when a softmax warp gave up
      if (elect_one()) mma_commit(&sh->drain);
      mbar_wait_warp(&sh->drain, 0, kDiffDrainNs);
    }
  } else if (warp >= 4) {
    const int m = (warp - 4) >> 2;  // the map
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_addr = lane_addr + C::TM_S + 128 * m, o_addr = lane_addr + C::TM_O + 128 * m;
    const uint64_t c2 = f32x2_pack(scale_log2, scale_log2);
    float m_ref = -INFINITY, l = 0.f, lx = 0.f;  // (lx: for the log-sum-exp)
    bool ok = limit_ns != 0;
    for (int u = 0; u < steps; ++u) {
      const uint32_t buf = s_addr + 64 * (u & 1);
      const int valid = u + 1 == steps ? last - 64 * (u & 1) : 64;  // real keys of the step
      mbar_await(&sh->s_full[m][u & 1], (uint32_t)((u >> 1) & 1), polls, ok);
      tc_fence_after();
      // The reference is the first step's maximum, and later steps' exponentials
      // are taken against it without looking for their own: fp32 and bf16 hold p
      // and its sums up to far above 2^24, and a row's precision does not depend
      // on their common factor.  Only when a step's sum or one weight passes 2^24 does the row
      // take the step's maximum as its new reference, with O and l scaled down and
      // the exponentials taken again (the scores are still there).  So does a row
      // whose scores were all -inf so far: it has no reference yet, and its weights of
      // 0 are taken against 0.
      if (u == 0) m_ref = row_max(buf, valid);
      uint32_t pk[32];
      float top, rx;
      float rs = softmax_pass<TRAIN>(buf, valid, c2, m_ref == -INFINITY ? 0.f : -m_ref * scale_log2, pk, top, rx);
      const bool grown = !(rs <= kDiffGrown && top <= kDiffGrownLog2 && m_ref > -INFINITY);
      if (__any_sync(0xffffffffu, grown)) {
        const float mt = row_max(buf, valid);
        float alpha = 1.f;
        if (grown && mt > -INFINITY) {
          alpha = ex2_approx((m_ref - mt) * scale_log2);  // (0 where there was none)
          m_ref = mt;
        }
        l *= alpha;
        lx *= alpha;
        if (u > 0) {
          mbar_await(&sh->pv_done[m], (uint32_t)((u - 1) & 1), polls, ok);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            tmem_ld32(o_addr + 32 * c, pk);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = __float_as_uint(__uint_as_float(pk[i]) * alpha);
            tmem_st32(o_addr + 32 * c, pk);
          }
        }
        rs = softmax_pass<TRAIN>(buf, valid, c2, m_ref == -INFINITY ? 0.f : -m_ref * scale_log2, pk, top, rx);
        if (top != top) rs = rx = top;  // a NaN among the scores is one of the row
      }
      l += rs;
      lx += rx;
      tmem_st32(buf, pk);  // over scores that have been read
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&sh->p_full[m][u & 1]);
    }
    if (n > 0) mbar_await(&sh->o_full, 0, polls, ok);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) diff_timeout(sh, status);
    const int row = qt * 128 + r;
    if (TRAIN && ok && row < N) {
      const size_t BH = gridDim.x / nb;
      lse[((size_t)m * BH + bh) * N + row] = n > 0 ? (m_ref * scale_log2 + log2f(lx)) * kLn2 : -INFINITY;
    }
    sh->sum[m][r] = m_ref == -INFINITY ? NAN : l;  // (kept keys that all score -inf: 0 / 0)
    named_bar_sync(1, 256);  // (reached by every softmax thread, after a time-out too)
    tc_fence_after();
    // features [m D/2, m D/2 + D/2) of this row: out = O_1 / l_1 - lam O_2 / l_2
    const float lh = lambda_of(lam, lam_bf16, h);
    const float i1 = n > 0 ? 1.f / sh->sum[0][r] : 0.f, i2 = n > 0 ? 1.f / sh->sum[1][r] : 0.f;
    if (n == 0) mbar_await(&sh->q_full, 0, polls, ok);  // the Q buffer is written over: its load must have landed
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int f0 = m * (D / 2) + 32 * c;  // 32 features
      uint32_t a[32], o2[32], pk[16], pk2[16];
      if (ok && n > 0) {
        tmem_ld32(lane_addr + C::TM_O + f0, a);
        tmem_ld32(lane_addr + C::TM_O + 128 + f0, o2);
        tmem_ld_wait();
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x0 = 0.f, x1 = 0.f, y0 = 0.f, y1 = 0.f;
        if (n > 0) {
          y0 = __uint_as_float(o2[2 * i]) * i2;
          y1 = __uint_as_float(o2[2 * i + 1]) * i2;
          x0 = fmaf(__uint_as_float(a[2 * i]), i1, -lh * y0);
          x1 = fmaf(__uint_as_float(a[2 * i + 1]), i1, -lh * y1);
        }
        pk[i] = pack_bf16x2(x0, x1);
        pk2[i] = pack_bf16x2(y0, y1);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t piece = (uint32_t)(f0 / 8 + t), at = (piece / 8) * 16384 + sw128_offset((uint32_t)r, piece % 8);
        st_shared_v4(sbase + C::OFF_Q + at, pk[4 * t], pk[4 * t + 1], pk[4 * t + 2], pk[4 * t + 3]);
        if (TRAIN) st_shared_v4(sbase + C::OFF_K + at, pk2[4 * t], pk2[4 * t + 1], pk2[4 * t + 2], pk2[4 * t + 3]);
      }
    }
    fence_proxy_async_smem();
    named_bar_sync(1, 256);
    if (warp == 4 && lane == 0 && !sh->abort_flag) {
      tma_store_4d(&tm_out, smem + C::OFF_Q, 0, qt * 128, h * C::DCH, b);
      if (TRAIN) tma_store_4d(&tm_out2, smem + C::OFF_K, 0, qt * 128, h * C::DCH, b);
      bulk_commit_group();
      bulk_wait_group_read0();
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

template <int D, bool TRAIN>
cudaError_t launch_diff_fwd_t(const DiffArgs& a, cudaStream_t s) {
  using C = DiffCfg<D>;
  cudaError_t e = cudaFuncSetAttribute(diff_fwd_kernel<D, TRAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  diff_fwd_kernel<D, TRAIN><<<a.B * a.heads * a.nb, kDiffThreads, C::SMEM, s>>>(
      *a.tm_q, *a.tm_k, *a.tm_v, *a.tm_out, *a.tm_out2, a.row_ptr, a.col_idx, a.lam, a.lam_bf16, a.lse, a.N, a.heads,
      a.nb, a.mask_per_bh, a.scale_log2, a.status, a.wait_limit_ns);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_forward(const DiffArgs& a, cudaStream_t s) {
  if (a.lse != nullptr) return a.d == 64 ? launch_diff_fwd_t<64, true>(a, s) : launch_diff_fwd_t<128, true>(a, s);
  return a.d == 64 ? launch_diff_fwd_t<64, false>(a, s) : launch_diff_fwd_t<128, false>(a, s);
}

}  // namespace salad
