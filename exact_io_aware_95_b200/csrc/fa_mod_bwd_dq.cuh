// dQ of the modified-score attention in a fixed order, for sm_100a: the dQ pass
// of the plain deterministic backward (fa_bwd_dq.cuh: one CTA per 128-row query
// tile and head walks its key tiles in increasing order, dQ summed in tensor
// memory) with the scores, mask plan and grouped heads of fa_mod_bwd.cuh.  The
// main kernel then runs without its dQ product and its atomics, and dQ, dK and
// dV are bitwise reproducible, for 7 instead of 5 matrix products per tile pair.
// A thread owns a query row: its interval masks the columns (only in tiles that
// some row of its warp sees in part) and its bias is taken column by column,
// exact in the distance.  dS is formed as in the main kernel, from
// P (1 - t^2) 2^15 in fp16.
//
// Bound like the plain pass (the P and dS chain of 256 threads beside three
// products a tile).  The whole call against the one with atomics, calls back to
// back: 1391-1397 us against 1069-1095 at 4 x 16(4) x 4096 x 128 causal capped, 370
// against 272 at 2 x 16 x 8192 x 64 with documents of 700 tokens and a bias, 96
// against 64 at 2 x 8(1) x 2047 x 64 with a window of 512, cap and bias.
#pragma once
#include "fa_bwd_dq.cuh"
#include "fa_mod_bwd.cuh"

namespace fa {

// bits [lo, hi) of 32 columns
__device__ __forceinline__ uint32_t chunk_bits(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  return (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & (lo == 32 ? 0u : 0xffffffffu << lo);
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(320, 1)
    fa_mod_bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                         const ModBwdParams p) {
  using C = DqCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ---- work item: (query tile i, batch entry, head), late tiles first (under a
  // causal mask the longest), heads side by side: a group's share K and V
  const int nbh = p.B * p.H;
  const int bh = blockIdx.x % nbh;
  const int i = p.T - 1 - blockIdx.x / nbh;
  const int h = bh % p.H, b = bh / p.H, hk = h / p.G;
  const int q0 = 128 * i;
  const PlanQTile* qt = p.plan.qt + static_cast<size_t>(b) * p.T + i;
  const int jb = max(qt->kbeg, 0), nkv = min(qt->kend, p.T) - jb;  // clamped as in the forward pass
  if (nkv <= 0) {  // a tile that sees nothing: uniform over the CTA, before any barrier or allocation
    uint4* dst = reinterpret_cast<uint4*>(p.dq) + ((static_cast<size_t>(b) * p.N + q0) * p.H + h) * (D / 8);
    for (int e = threadIdx.x; e < min(128, p.N - q0) * (D / 8); e += C::THREADS)
      dst[static_cast<size_t>(e / (D / 8)) * p.H * (D / 8) + e % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }

  auto bar = [&](int n) -> uint32_t { return sbase + C::OFF_BAR + 8u * n; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);

  if (threadIdx.x == 0) {
    mbar_init(bar(C::BAR_QDO), 1);
    for (int s = 0; s < C::NSTAGE; ++s) {
      mbar_init(bar(C::BAR_KV_FULL + s), 1);
      mbar_init(bar(C::BAR_KV_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(C::BAR_S + s), 1);
      mbar_init(bar(C::BAR_S_FREE + s), 256);
    }
    mbar_init(bar(C::BAR_DP), 1);
    mbar_init(bar(C::BAR_DP_FREE), 256);
    mbar_init(bar(C::BAR_DS), 256);
    mbar_init(bar(C::BAR_DS_EMPTY), 1);
    mbar_init(bar(C::BAR_ACC), 1);
    mbar_init(bar(C::BAR_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmdO);
      mbar_arrive_expect_tx(bar(C::BAR_QDO), 2 * C::TILE_BYTES);
      for (int c = 0; c < C::NCHUNK; ++c) {
        tma_load_4d(sbase + C::OFF_Q + c * 16384, &tmQ, bar(C::BAR_QDO), c * 64, h, q0, b);
        tma_load_4d(sbase + C::OFF_DO + c * 16384, &tmdO, bar(C::BAR_QDO), c * 64, h, q0, b);
      }
      int issued = 0;
      for (int j = 0; j < nkv; ++j) {
        const int st = j % C::NSTAGE;
        const uint32_t ph = (j / C::NSTAGE) & 1;
        if (!mbar_wait(bar(C::BAR_KV_EMPTY + st), ph ^ 1u, abort_flag)) break;
        mbar_arrive_expect_tx(bar(C::BAR_KV_FULL + st), 2 * C::TILE_BYTES);
        const uint32_t dst = sbase + C::OFF_KV + st * 2 * C::TILE_BYTES;
        for (int c = 0; c < C::NCHUNK; ++c) {
          tma_load_4d(dst + c * 16384, &tmK, bar(C::BAR_KV_FULL + st), c * 64, hk, 128 * (jb + j), b);
          tma_load_4d(dst + C::TILE_BYTES + c * 16384, &tmV, bar(C::BAR_KV_FULL + st), c * 64, hk, 128 * (jb + j), b);
        }
        ++issued;
      }
      if (*abort_flag) {  // let the copies in flight land before the CTA exits
        mbar_wait_drain(bar(C::BAR_QDO), 0);
        for (int n = 0; n < C::NSTAGE && n < issued; ++n) {
          const int m = issued - 1 - n;
          mbar_wait_drain(bar(C::BAR_KV_FULL + m % C::NSTAGE), (m / C::NSTAGE) & 1);
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false, false);  // S, dP
      constexpr uint32_t kIdQ = idesc_bf16_f32(128, D, false, true);     // dQ: B = K (MN-major view)
      const uint64_t dQ_k = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);      // Q, K-major A of S
      const uint64_t dO_k = sdesc_sw128(sbase + C::OFF_DO, 16, 1024);     // dO, K-major A of dP
      const uint64_t dKV_k = sdesc_sw128(sbase + C::OFF_KV, 16, 1024);    // K or V stage, K-major B of S / dP
      const uint64_t dK_mn = sdesc_sw128(sbase + C::OFF_KV, 16384, 1024); // K stage, MN-major B of dQ
      const uint64_t dS_k = sdesc_sw128(sbase + C::OFF_DS, 16, 1024);     // dS, K-major A of dQ
      constexpr uint32_t kStageAdv = (2 * C::TILE_BYTES) >> 4;
      constexpr uint32_t kTileAdv = C::TILE_BYTES >> 4;
      auto issue_s = [&](int j) {
        const uint64_t bk = dKV_k + (j % C::NSTAGE) * kStageAdv;
        const uint32_t dst = tmem + ((j & 1) ? C::TM_S1 : C::TM_S0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(dst, sdesc_adv(dQ_k, off), sdesc_adv(bk, off), kIdS, kk > 0);
        }
        umma_commit(bar(C::BAR_S + (j & 1)));
      };
      auto issue_dp = [&](int j) {
        const uint64_t bv = dKV_k + (j % C::NSTAGE) * kStageAdv + kTileAdv;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(tmem + C::TM_DP, sdesc_adv(dO_k, off), sdesc_adv(bv, off), kIdS, kk > 0);
        }
        umma_commit(bar(C::BAR_DP));
      };
      bool ok = mbar_wait(bar(C::BAR_QDO), 0, abort_flag) && mbar_wait(bar(C::BAR_KV_FULL), 0, abort_flag);
      if (ok) {
        tc_fence_after();
        issue_s(0);
        issue_dp(0);
      }
      for (int j = 0; ok && j < nkv; ++j) {
        if (j + 1 < nkv) {
          const int j1 = j + 1;
          if (!(ok = mbar_wait(bar(C::BAR_KV_FULL + j1 % C::NSTAGE), (j1 / C::NSTAGE) & 1, abort_flag))) break;
          // S(j+1) reuses the columns of S(j-1): wait until they were read
          if (j1 >= 2 && !(ok = mbar_wait(bar(C::BAR_S_FREE + (j1 & 1)), ((j1 >> 1) - 1) & 1, abort_flag))) break;
          tc_fence_after();
          issue_s(j1);
          // dP(j+1) overwrites dP(j): wait until it was read
          if (!(ok = mbar_wait(bar(C::BAR_DP_FREE), j & 1, abort_flag))) break;
          tc_fence_after();
          issue_dp(j1);
        }
        // dQ += dS(j) K(j)
        if (!(ok = mbar_wait(bar(C::BAR_DS), j & 1, abort_flag))) break;
        tc_fence_after();
        const uint64_t bk = dK_mn + (j % C::NSTAGE) * kStageAdv;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ss(tmem + C::TM_DQ, sdesc_adv(dS_k, (kk >> 2) * 16384 + (kk & 3) * 32), sdesc_adv(bk, kk * 2048), kIdQ,
                  (j > 0 || kk > 0));
        umma_commit(bar(C::BAR_KV_EMPTY + j % C::NSTAGE));
        umma_commit(bar(C::BAR_DS_EMPTY));
      }
      if (ok) umma_commit(bar(C::BAR_ACC));
      if (*abort_flag) {
        umma_commit(bar(C::BAR_DRAIN));
        mbar_wait_drain(bar(C::BAR_DRAIN), 0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ P, dS, epilogue
    const int w = warp >> 2;          // key columns 64w .. 64w+63 of every tile
    const int t = threadIdx.x & 127;  // query row within the tile == tensor-memory lane
    const int q = q0 + t;
    const bool row_ok = q < p.N;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    constexpr float kLog2e = 1.4426950408889634f;
    // Rows past the end: LSE = +inf makes their P (and dS) exactly 0.
    float lse2 = INFINITY, dvl = 0.f;
    int2 see = make_int2(0, 0);
    if (row_ok) {
      const size_t li = (static_cast<size_t>(b) * p.H + h) * p.N + q;
      lse2 = p.lse[li] * kLog2e;
      dvl = -p.dvec[li] / kDsUp;
      see = p.plan.rows[static_cast<size_t>(b) * p.N + q];
    }
    const float slope = BIAS ? slope_log2(p.slopes[h]) : 0.f;
    const uint64_t y2 = CAP ? f2_pack(p.cap_log2, p.cap_log2) : f2_pack(p.scale_log2, p.scale_log2);
    const uint64_t up = f2_pack(kDsUp, kDsUp), down = f2_pack(-kDsUp, -kDsUp), dn = f2_pack(1.f / kDsUp, 1.f / kDsUp);
    const uint32_t region = sbase + C::OFF_DS + w * 16384;  // keys 64w..64w+63 of dS
    bool ok = true;
    for (int j = 0; j < nkv; ++j) {
      const int k0 = 128 * (jb + j);
      ok = mbar_wait(bar(C::BAR_S + (j & 1)), (j >> 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tm_s = (j & 1) ? C::TM_S1 : C::TM_S0;
      const bool edge = __any_sync(0xffffffffu, k0 < see.x || k0 + 128 > see.y);
      uint32_t pk[2][16];
#pragma unroll
      for (int hc = 0; hc < 2; ++hc) {
        const int cc = 2 * w + hc;  // 32-key chunk of the tile
        uint32_t s[32];
        tmem_ld32(lane_base + tm_s + 32 * cc, s);
        tmem_wait_ld(s);
        if constexpr (CAP) cap_scores(s, p.x_mul);
        float dist = static_cast<float>(q - k0 - 32 * cc);
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const uint64_t s2 = f2_pack(__uint_as_float(s[2 * m]), __uint_as_float(s[2 * m + 1]));
          float x0, x1, a0, a1;
          float l0 = -lse2, l1 = -lse2;
          if constexpr (BIAS) {
            l0 = fmaf(-slope, fabsf(dist), l0);
            l1 = fmaf(-slope, fabsf(dist - 1.f), l1);
            dist -= 2.f;
          }
          f2_unpack(ffma2(s2, y2, f2_pack(l0, l1)), x0, x1);
          const uint64_t pr = f2_pack(ex2(x0), ex2(x1));
          f2_unpack(fmul2(pr, CAP ? ffma2(fmul2(s2, down), s2, up) : up), a0, a1);
          pk[hc][m] = pack_f16x2(a0, a1);  // P (1 - t^2) 2^15
        }
        if (edge) {  // pairs outside the mask: 0 whatever they hold
          const uint32_t seen = chunk_bits(see.x - k0 - 32 * cc, see.y - k0 - 32 * cc);
#pragma unroll
          for (int m = 0; m < 16; ++m)
            pk[hc][m] &= ((seen >> (2 * m)) & 1u ? 0xffffu : 0u) | ((seen >> (2 * m + 1)) & 1u ? 0xffff0000u : 0u);
        }
      }
      tc_fence_before();
      mbar_arrive(bar(C::BAR_S_FREE + (j & 1)));
      ok = mbar_wait(bar(C::BAR_DP), j & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t dp[2][32];
      tmem_ld32(lane_base + C::TM_DP + 32 * (2 * w), dp[0]);
      tmem_ld32(lane_base + C::TM_DP + 32 * (2 * w + 1), dp[1]);
      tmem_wait_ld(dp[0]);
      tmem_wait_ld(dp[1]);
      tc_fence_before();
      mbar_arrive(bar(C::BAR_DP_FREE));
      // the dS buffer is free once dQ(j-1) has consumed it
      ok = mbar_wait(bar(C::BAR_DS_EMPTY), (j & 1) ^ 1u, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int hc = 0; hc < 2; ++hc) {
        uint32_t wv[16];
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&pk[hc][m]));
          float d0, d1;
          const uint64_t dpm = f2_pack(__uint_as_float(dp[hc][2 * m]), __uint_as_float(dp[hc][2 * m + 1]));
          f2_unpack(fmul2(f2_pack(g.x, g.y), ffma2(dpm, dn, f2_pack(dvl, dvl))), d0, d1);
          wv[m] = pack_bf16x2(d0, d1);
        }
        // 32 keys -> 16-byte chunks hc*4 + 0..3 of row t in region w
#pragma unroll
        for (int u = 0; u < 4; ++u)
          st_shared_v4(region + sw128_offset(t, hc * 4 + u), wv[4 * u], wv[4 * u + 1], wv[4 * u + 2], wv[4 * u + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bar(C::BAR_DS));
    }
    // epilogue: dQ = bf16(scale * acc); warpgroup w stores columns w*D/2 ..
    if (ok) {
      ok = mbar_wait(bar(C::BAR_ACC), 0, abort_flag);
      if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        const size_t row = (static_cast<size_t>(b) * p.N + q) * p.H + h;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.dq) + row * D;
        const float sc = p.scale;
#pragma unroll 1
        for (int cc = w * (D / 64); cc < (w + 1) * (D / 64); ++cc) {
          uint32_t a[32];
          tmem_ld32(lane_base + C::TM_DQ + 32 * cc, a);
          tmem_wait_ld(a);
          uint32_t wv[16];
#pragma unroll
          for (int n = 0; n < 16; ++n)
            wv[n] = pack_bf16x2(__uint_as_float(a[2 * n]) * sc, __uint_as_float(a[2 * n + 1]) * sc);
          if (row_ok) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              st_global_v4(dst + 32 * cc + 8 * u, wv[4 * u], wv[4 * u + 1], wv[4 * u + 2], wv[4 * u + 3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace fa
