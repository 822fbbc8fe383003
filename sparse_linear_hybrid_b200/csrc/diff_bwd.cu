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
//                     whole tiles (pad rows: 1e30, finite, for p = 0)
//   diff_dq_kernel    one CTA per (query tile, b, h), 64 keys a step in two buffers
//                     of tensor memory: S_1, S_2 and dP, then dS_1 and dS_2 as bf16
//                     over S_1; one thread a row and half of the step's keys; and
//                     the CTA's share of dlam, in fp32 from p and dp themselves
//   diff_dkdv_kernel  one CTA per (key tile, b, h) over the query tiles that keep
//                     it, 64 queries a step: S_1^T, S_2^T and dP^T are read into
//                     registers and replaced by the next step's at once; (P_1 -
//                     lam P_2)^T and dS_1^T go to tensor memory, dS_2^T, for which
//                     no columns are left beside the 256 of dV and dK, to shared
//                     memory.  The products of a step so run beside the row
//                     warps' work on the one before and after it
//   diff_dlam_kernel  sums the shares of every head in a fixed order
// Gradients are rounded once, to bf16 (dlam to lam's type).  P and dS enter their
// products as bf16, a choice: half a step of each weight, averaged over the sum.
// Of one 9,360-token step of 12 heads of 128 (forward and backward 1,047 us, 1,091 in a
// long run) the prep takes 22 us, dQ 327, dK/dV 395, by themselves; the tensor cores are
// busy 45 and 49 % of that.  dK/dV is bound by shared memory (its products read
// both operands from there, dS_2^T passes through it), dQ by the row warps, the prep
// by its instructions (it issues in 66 % of the cycles, at 49 % of DRAM's rate).  One
// pair of exponentials in four on the FMA pipe (949 us; none 955, one in two 986).
// Warp roles, 384 threads: warp 0 TMA producer, warps 1-3 tcgen05 issuers (warp 1 owns the tensor
// memory), warps 4-11 the rows (TMEM lane quarter = warp % 4).  There are several
// issuers because a warp that pushes products into a full tensor-core queue holds
// up the shared-memory instructions of its scheduler's other warps: with one
// issuer two of the eight row warps ran 500 to 900 of 2,400 cycles a step behind
// the others (clock64).  Every barrier wait is bounded; on a time-out the kernel
// records it and drains.
#include "diff.cuh"
#include "internal.h"

namespace salad {
namespace {

constexpr int kDiffBwdThreads = 384;
constexpr uint64_t kDiffBwdDrainNs = 1000000000ull;
constexpr float kDiffLog2e = 1.4426950408889634f;
constexpr float kDiffPadLse = 1e30f;

struct DiffBwdShared {
  uint64_t fixed_full;
  uint64_t ring_full[4], ring_empty[4];                   // dK/dV kernel
  uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];  // dQ kernel
  uint64_t buf_full[2], buf_read[2], buf_ds[2], buf_done[2];  // dQ kernel, per buffer
  uint64_t s_full, s_read, ds_full, mm_done;               // dK/dV kernel
  uint64_t drain;
  uint32_t tmem_base;
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
  // dK/dV kernel: four stages of 64 rows of Q, dO and the four row vectors; dS_2^T
  static constexpr int HALF = 64 * D * 2;  // DCH chunks of 8 KB
  static constexpr int STAGES = 4;
  static constexpr int VEC = 4 * 64 * 4;
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_DS = OFF_RING + STAGES * 2 * HALF;
  static constexpr int OFF_VEC = OFF_DS + 16384;
  static constexpr int OFF_BAR = OFF_VEC + STAGES * VEC;
  static constexpr int USED = OFF_BAR + (int)sizeof(DiffBwdShared) + 1024;
  static constexpr int SMEM = USED > 122880 ? USED : 122880;
  static constexpr uint32_t IDESC_SH = idesc_bf16(128, 64, false, false);  // 64 keys or queries
  static constexpr uint32_t IDESC_H = idesc_bf16(128, 64, false, true);    // gradient of one half of q or k
  static constexpr uint32_t IDESC_V = idesc_bf16(128, D, false, true);
  static_assert(DQ_SMEM <= 232448 && SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void diff_bwd_timeout(uint32_t* status) { atomicOr(status, kStatusTimeout); }

// K-steps [first, first + count) of X Y^T into D, both K-major: 128-byte rows in
// 64-feature chunks, X's of 128 rows, Y's of y_chunk bytes; the first one overwrites.
template <int COUNT>
__device__ __forceinline__ void mma_steps(uint32_t d_tmem, uint32_t x, uint32_t y, int first, uint32_t idesc,
                                          int y_chunk = 16384) {
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    const int f = first + i;
    mma_bf16_ss(d_tmem, sw128_desc(x + (f / 4) * 16384 + (f % 4) * 32, 16, 1024),
                sw128_desc(y + (f / 4) * y_chunk + (f % 4) * 32, 16, 1024), idesc, i > 0 ? 1u : 0u);
  }
}

// rows[B*Hh][npad/64][4][64]: lse_1 and lse_2 (base 2; kDiffPadLse in pad rows), D_1, D_2
// of 64 queries, the piece that a step of the dK/dV kernel loads.
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
  const int64_t bh = (int64_t)b * heads + h;
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
    float* at = rows + bh * npad * 4 + n / 64 * 256 + n % 64;
    at[0] = n < N ? lse[bh * N + n] * kDiffLog2e : kDiffPadLse;
    at[64] = n < N ? lse[(BH + bh) * N + n] * kDiffLog2e : kDiffPadLse;
    at[128] = fmaf(lambda_of(lam, lam_bf16, h), d2, d0);
    at[192] = d2;
  }
}

__device__ __forceinline__ uint64_t pair_of(const uint32_t (&s)[32], int i) {
  return f32x2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
  float a, b;
  f32x2_unpack(v, a, b);
  return pack_bf16x2(a, b);
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
  // A step is 64 keys.  Two buffers of 192 columns, each S_1 [0,64), S_2 [64,128) and
  // dP [128,192) of a step; a thread's half e of the keys is columns [32 e, +32) of
  // each, and it writes dS_1 as bf16 over [32 e, +16) and dS_2 over [32 e + 16, +16)
  // once it holds all three in registers.  dQ_1 [384,448), dQ_2 [448,512).  At d = 64
  // the two products take both halves of k (N = 64) and the half that does not
  // belong is left aside.
  constexpr uint32_t TM_BUF = 192, TM_DP = 128, TM_DQ = 384;
  extern __shared__ uint8_t diff_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(diff_smem_raw) + 1023) & ~uintptr_t(1023));
  DiffBwdShared* sh = reinterpret_cast<DiffBwdShared*>(smem + C::DQ_OFF_BAR);
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
    mbar_init(&sh->fixed_full, 1);
    for (int st = 0; st < 3; ++st) mbar_init(&sh->k_full[st], 1), mbar_init(&sh->k_empty[st], 1);
    for (int st = 0; st < 2; ++st) mbar_init(&sh->v_full[st], 1), mbar_init(&sh->v_empty[st], 1);
    for (int f = 0; f < 2; ++f) {
      mbar_init(&sh->buf_full[f], 2);  // S_1, and S_2 with dP
      mbar_init(&sh->buf_read[f], 8);
      mbar_init(&sh->buf_ds[f], 8);
      mbar_init(&sh->buf_done[f], 1);
    }
    mbar_init(&sh->drain, 3);
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
  const uint32_t q_s = sbase + C::OFF_FIX, do_s = q_s + C::TILE;

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      bool ok = true;
      int kl = 0, vl = 0;  // K and V loads issued
      mbar_arrive_expect_tx(&sh->fixed_full, 2 * C::TILE);
      tma_load_4d(smem + C::OFF_FIX, &tm_q, &sh->fixed_full, 0, qt * 128, h * C::DCH, b);
      tma_load_4d(smem + C::OFF_FIX + C::TILE, &tm_do, &sh->fixed_full, 0, qt * 128, h * C::DCH, b);
      // K_j is free once the gradient products of tile j have read it, V_j once dP_j is done
      for (int j = 0; j < n; ++j) {
        const int col = col_idx[c0 + j], ks = j % 3, vs = j & 1;
        if (!mbar_await_one(&sh->k_empty[ks], (uint32_t)((j / 3) & 1) ^ 1, limit_ns)) { ok = false; break; }
        mbar_arrive_expect_tx(&sh->k_full[ks], C::TILE);
        tma_load_4d(smem + C::DQ_OFF_K + ks * C::TILE, &tm_k, &sh->k_full[ks], 0, col * 128, h * C::DCH, b);
        ++kl;
        if (!mbar_await_one(&sh->v_empty[vs], (uint32_t)((j >> 1) & 1) ^ 1, limit_ns)) { ok = false; break; }
        mbar_arrive_expect_tx(&sh->v_full[vs], C::TILE);
        tma_load_4d(smem + C::DQ_OFF_V + vs * C::TILE, &tm_v, &sh->v_full[vs], 0, col * 128, h * C::DCH, b);
        ++vl;
      }
      if (!ok) diff_bwd_timeout(status);
      // every copy this thread started lands before the CTA exits
      mbar_wait(&sh->fixed_full, 0, kDiffBwdDrainNs);
      for (int i = (kl > 3 ? kl - 3 : 0); i < kl; ++i)
        mbar_wait(&sh->k_full[i % 3], (uint32_t)((i / 3) & 1), kDiffBwdDrainNs);
      for (int i = (vl > 2 ? vl - 2 : 0); i < vl; ++i)
        mbar_wait(&sh->v_full[i & 1], (uint32_t)((i >> 1) & 1), kDiffBwdDrainNs);
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------- tcgen05 issuers: S_2 and dP of
    // a step (warp 2) once the row warps hold those of two steps before in registers,
    // S_1 (warp 1), whose columns dS took, once the gradient products (warp 3) have
    // read that
    if (n > 0) {  // (whole warps; one lane issues)
      bool ok = limit_ns != 0;
      mbar_await(&sh->fixed_full, 0, polls, ok);
      int ks = 0;
      uint32_t kph = 0;  // K stage and its parity
      for (int u = 0; u < steps; ++u) {
        const int f = u & 1, vs = (u >> 1) & 1;
        const uint32_t ph = (uint32_t)((u >> 1) & 1), buf = tmem + TM_BUF * f, rows64 = 8192u * f;
        const bool last_use = f == 1 || u + 1 == steps;  // of the step's key tile
        mbar_await(&sh->k_full[ks], kph, polls, ok);
        if (warp == 2) mbar_await(&sh->v_full[vs], (uint32_t)((u >> 2) & 1), polls, ok);
        if (warp == 3)
          mbar_await(&sh->buf_ds[f], ph, polls, ok);
        else if (u >= 2)
          mbar_await(warp == 1 ? &sh->buf_done[f] : &sh->buf_read[f], ph ^ 1, polls, ok);
        tc_fence_after();
        const uint32_t kt = sbase + C::DQ_OFF_K + ks * C::TILE + rows64;
        if (warp == 1) {
          if (elect_one() && ok) {
            mma_steps<D / 32>(buf, q_s, kt, 0, C::IDESC_SH);
            mma_commit(&sh->buf_full[f]);
          }
        } else if (warp == 2) {
          if (elect_one() && ok) {
            mma_steps<D / 32>(buf + 64, q_s, kt, D / 32, C::IDESC_SH);
            mma_steps<D / 16>(buf + TM_DP, do_s, sbase + C::DQ_OFF_V + vs * C::TILE + rows64, 0, C::IDESC_SH);
            mma_commit(&sh->buf_full[f]);
            if (last_use) mma_commit(&sh->v_empty[vs]);
          }
        } else if (elect_one() && ok) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(tmem + TM_DQ + 64 * m, buf + 32 * (kk >> 1) + 16 * m + 8 * (kk & 1),
                          sw128_desc(kt + (C::DCH == 2 ? m * 16384 : 0) + kk * 2048, 16384, 1024), C::IDESC_H,
                          (u > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&sh->buf_done[f]);
          if (last_use) mma_commit(&sh->k_empty[ks]);  // (S of this step ended before the row warps formed dS)
        }
        if (f == 1) {
          ks = ks == 2 ? 0 : ks + 1;
          kph = ks == 0 ? kph ^ 1 : kph;
        }
      }
      if (!__all_sync(0xffffffffu, ok)) diff_bwd_timeout(status);
      // every product has ended before the tensor memory is given back, also when a row warp gave up
      if (elect_one()) mma_commit(&sh->drain);
      mbar_wait_warp(&sh->drain, 0, kDiffBwdDrainNs);
    }
  } else {
    // one thread a query row and half of the keys of every tile
    const int quarter = warp & 3, r = quarter * 32 + lane, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    const float* at = rows + ((size_t)bh * npad + qt * 128 + (r & 64)) * 4 + (r & 63);
    const float l1 = at[0], l2 = at[64], D1 = at[128], D2 = at[192];
    const uint64_t c2 = f32x2_pack(scale_log2, scale_log2), nl1 = f32x2_pack(-l1, -l1), nl2 = f32x2_pack(-l2, -l2);
    const uint64_t nd1 = f32x2_pack(-D1, -D1), nd2 = f32x2_pack(-D2, -D2);
    uint64_t dl2 = 0;  // (0, 0)
    bool ok = limit_ns != 0;
    for (int u = 0; u < steps; ++u) {
      const int f = u & 1;
      const uint32_t buf = lane_addr + TM_BUF * f + 32 * half;
      mbar_await(&sh->buf_full[f], (uint32_t)((u >> 1) & 1), polls, ok);
      tc_fence_after();
      uint32_t s1[32], s2[32], g[32];
      tmem_ld32(buf, s1);
      tmem_ld32(buf + 64, s2);
      tmem_ld32(buf + TM_DP, g);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&sh->buf_read[f]);
      if (u + 1 == steps) {  // (only the last step can be short)
        const int valid = last - 64 * f - 32 * half;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i >= valid) s1[i] = s2[i] = __float_as_uint(-INFINITY);
      }
      uint32_t a[16], z[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint64_t x1 = f32x2_fma(pair_of(s1, k), c2, nl1), x2 = f32x2_fma(pair_of(s2, k), c2, nl2);
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
        const uint64_t p = f32x2_pack(p0, p1), q = f32x2_pack(q0, q1), gi = pair_of(g, k);
        a[k] = pack_pair(f32x2_mul(p, f32x2_add(gi, nd1)));
        z[k] = pack_pair(f32x2_mul(q, f32x2_add(gi, nd2)));
        dl2 = f32x2_fma(q, gi, dl2);
      }
      tmem_st16(buf, a);
      tmem_st16(buf + 16, z);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&sh->buf_ds[f]);
    }
    // the last gradient products (those of the step before them came first)
    if (n > 0) mbar_await(&sh->buf_done[(steps - 1) & 1], (uint32_t)(((steps - 1) >> 1) & 1), polls, ok);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      diff_bwd_timeout(status);
    } else {
      tc_fence_after();
      const int row = qt * 128 + r;
      const float mul = half ? -lambda_of(lam, lam_bf16, h) * scale : scale;  // half: the map whose dq this thread writes
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
    float dl, dl_odd;
    f32x2_unpack(dl2, dl, dl_odd);
    dl = qt * 128 + r < N ? dl + dl_odd : 0.f;  // (a row behind the last: 0 times an infinite key is NaN)
#pragma unroll
    for (int o = 16; o > 0; o /= 2) dl += __shfl_xor_sync(0xffffffffu, dl, o);
    if (lane == 0) sh->part[warp - 4] = dl;
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
  // 64 queries a step.  S_1^T [0,64), S_2^T [64,128), dP^T [128,192), dV
  // [192,192+d), dK_1 [320,384), dK_2 [384,448) (at d = 64 both halves of q, as in
  // the dQ kernel), (P_1 - lam P_2)^T [448,480) and dS_1^T [480,512) as bf16;
  // a thread's half e of the queries is columns [32 e, +32) of the scores and dP^T
  // and [16 e, +16) of the bf16 operands.
  constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 192, TM_DK = 320, TM_A = 448, TM_DS = 480;
  extern __shared__ uint8_t diff_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(diff_smem_raw) + 1023) & ~uintptr_t(1023));
  DiffBwdShared* sh = reinterpret_cast<DiffBwdShared*>(smem + C::OFF_BAR);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t polls = polls_of(limit_ns);
  const int warp = warp_uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int kt = blockIdx.x % nb, bh = blockIdx.x / nb, b = bh / heads, h = bh % heads;
  const int mrow = (mask_per_bh ? bh : h) * nb + kt;
  const int mask_rows = (mask_per_bh ? (int)(gridDim.x / nb) : heads) * nb;
  const int c0 = warp_uniform(t_row_ptr[mrow]);
  const int n = warp_uniform(
      debug_row_ok(t_row_ptr, t_col_idx, mrow, mask_rows, nb, true, status) ? t_row_ptr[mrow + 1] - c0 : 0);

  if (threadIdx.x == 0) {
    mbar_init(&sh->fixed_full, 1);
    for (int s = 0; s < C::STAGES; ++s) mbar_init(&sh->ring_full[s], 1), mbar_init(&sh->ring_empty[s], 1);
    mbar_init(&sh->s_full, 2);  // the scores and dP^T
    mbar_init(&sh->s_read, 8);
    mbar_init(&sh->ds_full, 8);
    mbar_init(&sh->mm_done, 1);
    mbar_init(&sh->drain, 3);
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
  const uint32_t k_s = sbase + C::OFF_FIX, v_s = k_s + C::TILE;

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      bool ok = true;
      int loads = 0;
      mbar_arrive_expect_tx(&sh->fixed_full, 2 * C::TILE);
      tma_load_4d(smem + C::OFF_FIX, &tm_k, &sh->fixed_full, 0, kt * 128, h * C::DCH, b);
      tma_load_4d(smem + C::OFF_FIX + C::TILE, &tm_v, &sh->fixed_full, 0, kt * 128, h * C::DCH, b);
      // step i: rows [64 (i & 1), + 64) of query tile i / 2, into the stage that
      // the gradient products of step i - 4 have read
      int qi = 0;
      for (int i = 0; i < 2 * n; ++i) {
        if ((i & 1) == 0) qi = t_col_idx[c0 + (i >> 1)];
        const int s = i % C::STAGES, q0 = qi * 128 + 64 * (i & 1);
        if (!mbar_await_one(&sh->ring_empty[s], (uint32_t)((i / C::STAGES) & 1) ^ 1, limit_ns)) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + C::OFF_RING + s * 2 * C::HALF;
        float* vec = reinterpret_cast<float*>(smem + C::OFF_VEC + s * C::VEC);
        mbar_arrive_expect_tx(&sh->ring_full[s], 2 * C::HALF + C::VEC);
        tma_load_4d(dst, &tm_q, &sh->ring_full[s], 0, q0, h * C::DCH, b);
        tma_load_4d(dst + C::HALF, &tm_do, &sh->ring_full[s], 0, q0, h * C::DCH, b);
        bulk_load(vec, rows + ((size_t)bh * npad + (size_t)q0) * 4, C::VEC, &sh->ring_full[s]);
        ++loads;
      }
      if (!ok) diff_bwd_timeout(status);
      // every copy this thread started lands before the CTA exits
      mbar_wait(&sh->fixed_full, 0, kDiffBwdDrainNs);
      for (int i = (loads > C::STAGES ? loads - C::STAGES : 0); i < loads; ++i)
        mbar_wait(&sh->ring_full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), kDiffBwdDrainNs);
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------- tcgen05 issuers: S^T of both
    // maps (warp 1) and dP^T (warp 2) of a step as soon as the row warps hold the
    // ones before in registers, the gradient products (warp 3) once their operands
    // are written
    if (n > 0) {  // (whole warps; one lane issues)
      bool ok = limit_ns != 0;
      mbar_await(&sh->fixed_full, 0, polls, ok);
      for (int i = 0; i < 2 * n; ++i) {
        const int s = i % C::STAGES;
        const uint32_t qs = sbase + C::OFF_RING + s * 2 * C::HALF;
        mbar_await(&sh->ring_full[s], (uint32_t)((i / C::STAGES) & 1), polls, ok);
        if (warp == 3)
          mbar_await(&sh->ds_full, (uint32_t)(i & 1), polls, ok);
        else if (i > 0)
          mbar_await(&sh->s_read, (uint32_t)((i - 1) & 1), polls, ok);
        tc_fence_after();
        if (warp == 1) {
          if (elect_one() && ok) {
            mma_steps<D / 32>(tmem + TM_S, k_s, qs, 0, C::IDESC_SH, 8192);
            mma_steps<D / 32>(tmem + TM_S + 64, k_s, qs, D / 32, C::IDESC_SH, 8192);
            mma_commit(&sh->s_full);
          }
        } else if (warp == 2) {
          if (elect_one() && ok) {
            mma_steps<D / 16>(tmem + TM_DP, v_s, qs + C::HALF, 0, C::IDESC_SH, 8192);
            mma_commit(&sh->s_full);
          }
        } else if (elect_one() && ok) {
          const uint32_t ds_s = sbase + C::OFF_DS;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t acc = (i > 0 || kk > 0) ? 1u : 0u;
            mma_bf16_ts(tmem + TM_DV, tmem + TM_A + 8 * kk, sw128_desc(qs + C::HALF + kk * 2048, 8192, 1024), C::IDESC_V, acc);
            mma_bf16_ts(tmem + TM_DK, tmem + TM_DS + 8 * kk, sw128_desc(qs + kk * 2048, 8192, 1024), C::IDESC_H, acc);
            mma_bf16_ss(tmem + TM_DK + 64, sw128_desc(ds_s + kk * 32, 16, 1024),
                        sw128_desc(qs + (C::DCH == 2 ? 8192 : 0) + kk * 2048, 8192, 1024), C::IDESC_H, acc);
          }
          mma_commit(&sh->mm_done);
          mma_commit(&sh->ring_empty[s]);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) diff_bwd_timeout(status);
      // every product has ended before the tensor memory is given back, also when a row warp gave up
      if (elect_one()) mma_commit(&sh->drain);
      mbar_wait_warp(&sh->drain, 0, kDiffBwdDrainNs);
    }
  } else {
    // one thread a key row and half of a step's queries
    const int quarter = warp & 3, r = quarter * 32 + lane, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    const float lh = lambda_of(lam, lam_bf16, h);
    const uint64_t c2 = f32x2_pack(scale_log2, scale_log2), nlam = f32x2_pack(-lh, -lh);
    const uint64_t minus = f32x2_pack(-1.f, -1.f), zero = f32x2_pack(0.f, 0.f);
    bool ok = limit_ns != 0;
    for (int i = 0; i < 2 * n; ++i) {
      const int s = i % C::STAGES;
      mbar_await(&sh->s_full, (uint32_t)(i & 1), polls, ok);
      mbar_await(&sh->ring_full[s], (uint32_t)((i / C::STAGES) & 1), polls, ok);
      tc_fence_after();
      const uint32_t vec = sbase + C::OFF_VEC + s * C::VEC + 128 * half;  // lse_1, then + 256 bytes lse_2, D_1, D_2
      uint32_t s1[32], s2[32], g[32];
      tmem_ld32(lane_addr + TM_S + 32 * half, s1);
      tmem_ld32(lane_addr + TM_S + 64 + 32 * half, s2);
      tmem_ld32(lane_addr + TM_DP + 32 * half, g);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&sh->s_read);
      uint32_t a[16], z1[16], z2[16];
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        uint32_t w[4][4];  // the row vectors of four queries
#pragma unroll
        for (int x = 0; x < 4; ++x) ld_shared_v4(vec + 256 * x + 8 * k, w[x][0], w[x][1], w[x][2], w[x][3]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          auto row = [&](int x) { return f32x2_pack(__uint_as_float(w[x][2 * u]), __uint_as_float(w[x][2 * u + 1])); };
          const uint64_t x1 = f32x2_fma(pair_of(s1, k + u), c2, f32x2_mul(row(0), minus));
          const uint64_t x2 = f32x2_fma(pair_of(s2, k + u), c2, f32x2_mul(row(1), minus));
          float p0, p1, q0, q1;
          if (((k + u) & 3) == 3) {
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
          uint64_t p = f32x2_pack(p0, p1), q = f32x2_pack(q0, q1);
          const uint64_t gi = pair_of(g, k + u);
          if (((k + u) & 3) == 3) {
            // The cubic takes a NaN for a large negative exponent.  A query with one has
            // a log-sum-exp that is not finite, and 0 times that brings the NaN back
            // (dq and dk have it through D, dv has it from here).
            p = f32x2_fma(row(0), zero, p);
            q = f32x2_fma(row(1), zero, q);
          }
          a[k + u] = pack_pair(f32x2_fma(nlam, q, p));
          z1[k + u] = pack_pair(f32x2_mul(p, f32x2_fma(row(2), minus, gi)));
          z2[k + u] = pack_pair(f32x2_mul(q, f32x2_fma(row(3), minus, gi)));
        }
      }
      // the products of the step before have read the operands' places
      if (i > 0) mbar_await(&sh->mm_done, (uint32_t)((i - 1) & 1), polls, ok);
      tc_fence_after();
      tmem_st16(lane_addr + TM_A + 16 * half, a);
      tmem_st16(lane_addr + TM_DS + 16 * half, z1);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        st_shared_v4(sbase + C::OFF_DS + sw128_offset((uint32_t)r, (uint32_t)(4 * half + x)), z2[4 * x], z2[4 * x + 1],
                     z2[4 * x + 2], z2[4 * x + 3]);
      fence_proxy_async_smem();
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&sh->ds_full);
    }
    if (n > 0) mbar_await(&sh->mm_done, (uint32_t)((2 * n - 1) & 1), polls, ok);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      diff_bwd_timeout(status);
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
      *a.tm_q64, *a.tm_k, *a.tm_v, *a.tm_do64, a.t_row_ptr, a.t_col_idx, a.rows, a.lam, a.lam_bf16, a.dk, a.dv, a.N,
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
