// Modified-score attention, forward, for sm_100a:
//
//     x_ij = scale q_i . k_j
//     y_ij = cap tanh(x_ij / cap)                    (CAP)
//     z_ij = y_ij - slope_h |i - j|                  (BIAS)
//     O_i  = sum_j softmax_j(z_ij) v_j,  LSE_i = ln sum_j exp(z_ij)
//
// over the keys lo_i <= j < hi_i of the mask plan (fa_plan.cuh); query head h
// reads key head h / (H / Hkv).  A row that sees nothing gets O = 0,
// LSE = -inf.  Optionally a second output holds bf16(O - bf16(O)), the part of
// O that rounding loses: the backward pass needs D = dO . O more exactly than
// O in bf16 gives it where one key dominates a row (dP - D cancels there).
//
// The pipeline is that of the plain forward (fa_fwd.cuh): a work item is two
// 128-row query tiles sharing one K/V stream, warps 0-7 softmax, warp 8 loads
// and takes work items, warp 9 issues the tensor-core products, S, P and O in
// tensor memory.  What differs:
//   - each query tile has its own key-tile range [kbeg, kend) from the plan,
//     and joins the shared stream only inside it: tiles of other documents,
//     outside the window or above the diagonal are never loaded or multiplied;
//   - the softmax warps turn a score row into z (base 2) in registers.  tanh is
//     an odd polynomial x P(x^2) on |x| <= 1, fitted by least squares with
//     reweighting to an absolute error below 1e-7, evaluated on packed fp32
//     pairs: 9 packed operations per pair of scores on the FMA pipes, where
//     exp and a reciprocal would put two more operations per score on the MUFU
//     pipe that the exponentials already fill (16 per clock per SM).  A warp
//     whose tile has a score beyond the cap takes the exponential form for that
//     tile: 1 - 2 / (1 + e^2x);
//   - the distance bias is linear in j on either side of the diagonal, so on a
//     tile that lies on one side for all rows of a warp (for causal rows: every
//     tile) it is a packed FMA with the running distance i - j, which is exact;
//     only tiles that straddle the diagonal with both sides visible take |i - j|
//     element by element.  (A running product slope j with the row's part taken
//     into the maximum saves one operation per pair, but adds up 64 roundings at
//     the size of 128 slopes: 1e-6 of the logsumexp.)
// What bounds it is the chain of a score tile through one softmax warpgroup
// (load, tanh, maximum, exponentials, store), of which two run side by side: at
// 4 x 16(4) x 4096 x 128 causal, ncu sees 42% of the issue slots, 26% of the
// tensor pipe, 26% of MUFU and 24% of the FMA pipes busy.  That size takes 300-326
// us with neither cap nor bias (275 GFLOP: 843-916 TFLOP/s), 358-376 us with the
// bias, 473-481 us with the cap, by card, calls back to back.  Measured and not
// kept: the score row transformed in rolled 32-column steps through tensor memory
// (470 us capped, but 727 against 687 us biased at 16384 tokens); the maximum taken
// of the raw scores and tanh and exponential in one loop (509 against 493 us).
#pragma once
#include "fa_fwd.cuh"
#include "fa_plan.cuh"

namespace fa {

// tanh x = x P(x^2), |x| <= kTanhRange: coefficients of P in increasing order
// (fitted in float64 on 4001 points by iteratively reweighted least squares;
// the largest absolute error is 2.0e-8, 9.5e-8 when evaluated in fp32: at a cap
// of 50 that is 7e-6 in the exponent, below what the logsumexp keeps.  A range
// of 1.25 with as many terms has 4.5e-7).
constexpr float kTanhRange = 1.f;
constexpr int kTanhTerms = 7;
__device__ constexpr float kTanhP[kTanhTerms] = {0.9999997019767761f,   -0.33332130312919617f, 0.13319583237171173f,
                                                 -0.05326583608984947f, 0.019973279908299446f, -0.00595127884298563f,
                                                 0.0009637715993449092f};

// t = tanh of a packed pair x, |x| <= kTanhRange
__device__ __forceinline__ uint64_t tanh2_poly(uint64_t x) {
  const uint64_t u = fmul2(x, x);
  uint64_t r = f2_pack(kTanhP[kTanhTerms - 1], kTanhP[kTanhTerms - 1]);
#pragma unroll
  for (int k = kTanhTerms - 2; k >= 0; --k) r = ffma2(r, u, f2_pack(kTanhP[k], kTanhP[k]));
  return fmul2(r, x);
}
// tanh for any x (NaN stays NaN): 1 - 2 / (1 + e^2x); 1 / inf = 0 and e^-inf = 0
// give the limits.  The argument is x * 2 log2(e).
constexpr float kTwoLog2e = 2.885390081777926815f;
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// base + mul / (1 + 2^x2) of a packed pair: with (1, -2) the tanh
__device__ __forceinline__ uint64_t tanh2_any(uint64_t x2, uint64_t base, uint64_t mul) {
  float a, b;
  f2_unpack(x2, a, b);
  f2_unpack(fadd2(f2_pack(ex2(a), ex2(b)), f2_pack(1.f, 1.f)), a, b);
  return ffma2(f2_pack(rcp_approx(a), rcp_approx(b)), mul, base);
}

// slope log2(e).  Kept finite, so that a distance of 0 adds 0 where the product
// overflows (slopes beyond 2.36e38); NaN stays NaN.
__device__ __forceinline__ float slope_log2(float slope) {
  const float s = slope * 1.4426950408889634f;
  return fabsf(s) == INFINITY ? copysignf(3.402823466e38f, s) : s;
}

struct ModFwdParams {
  void* o;
  void* o_low;          // bf16(O - bf16(O)), or nullptr
  float* lse;
  const float* slopes;  // [H], BIAS
  PlanView plan;
  int B, N, H, G;       // G = H / Hkv query heads per key head
  int T;                // ceil(N / 128)
  int npairs;           // ceil(N / 256)
  float scale_log2;     // scale * log2(e)             (no cap)
  float x_mul;          // scale / cap                 (CAP)
  float cap_log2;       // cap * log2(e)               (CAP)
};

struct ModFwdItem {
  int h, b, row0;
  int lo0, hi0, lo1, hi1;  // key tiles of the two query tiles
  int jb, je;              // the shared stream
  __device__ __forceinline__ int lo(int k) const { return k ? lo1 : lo0; }
  __device__ __forceinline__ int hi(int k) const { return k ? hi1 : hi0; }
};

__device__ __forceinline__ void mod_fwd_item(const ModFwdParams& p, int c, ModFwdItem& it) {
  // late query blocks first over the whole batch (under a causal mask the
  // longest), heads side by side: the heads of a group share K and V.  L2-sized
  // groups of heads, as in the plain forward, were equal or up to 5% slower.
  const int nbh = p.B * p.H;
  const int bh = c % nbh;
  const int pair = p.npairs - 1 - c / nbh;
  it.h = bh % p.H;
  it.b = bh / p.H;
  it.row0 = pair * 256;
  const PlanQTile* qt = p.plan.qt + static_cast<size_t>(it.b) * p.T + 2 * pair;
  const int2 r0 = *reinterpret_cast<const int2*>(qt);  // kbeg, kend
  const int2 r1 = 2 * pair + 1 < p.T ? *reinterpret_cast<const int2*>(qt + 1) : make_int2(0, 0);
  // clamped, so that a plan buffer that was never filled gives wrong numbers but
  // no access outside the tensors
  it.lo0 = max(r0.x, 0);
  it.hi0 = min(r0.y, p.T);
  it.lo1 = max(r1.x, 0);
  it.hi1 = min(r1.y, p.T);
  const bool a0 = it.lo0 < it.hi0, a1 = it.lo1 < it.hi1;
  it.jb = a0 ? (a1 ? min(it.lo0, it.lo1) : it.lo0) : (a1 ? it.lo1 : 0);
  it.je = max(a0 ? it.hi0 : 0, a1 ? it.hi1 : 0);
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1)
    fa_mod_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const ModFwdParams p) {
  using C = FwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + C::MISC_ABORT);
  volatile int* item_ring = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + C::MISC_ITEM);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + C::MISC_TMEM);
  const uint32_t resp = sbase + C::OFF_MISC + C::MISC_RESP;

  if (threadIdx.x == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar(C::BAR_Q + k), 1);
      mbar_init(bar(C::BAR_QFREE + k), 1);
      mbar_init(bar(C::BAR_S + k), 1);
      mbar_init(bar(C::BAR_OFIN + k), 1);
      mbar_init(bar(C::BAR_P + 2 * k), 128);
      mbar_init(bar(C::BAR_P + 2 * k + 1), 128);
      mbar_init(bar(C::BAR_ITEM_FULL + k), 1);
      mbar_init(bar(C::BAR_ITEM_EMPTY + k), C::ITEM_CONSUMERS);
    }
    for (int s = 0; s < C::NSTAGE; ++s) {
      mbar_init(bar(C::BAR_KV_FULL + s), 1);
      mbar_init(bar(C::BAR_KV_EMPTY + s), 1);
    }
    mbar_init(bar(C::BAR_CLC), 1);
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
  if (warp >= 8) {
    regs_set<104, kLaunchRegs>();
  }
  if (warp == 8) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      int item = blockIdx.x;
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      int nq[2] = {0, 0};
      uint32_t clc_phase = 0;
      bool clc_pending = false;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int slot = n & 1;
        if (n >= 2 && !(ok = mbar_wait(bar(C::BAR_ITEM_EMPTY + slot), ((n >> 1) - 1) & 1, abort_flag))) break;
        item_ring[slot] = item;
        mbar_arrive(bar(C::BAR_ITEM_FULL + slot));
        if (item < 0) break;
        ModFwdItem I;
        mod_fwd_item(p, item, I);
        const int hk = I.h / p.G;
        for (int k = 0; ok && k < 2; ++k) {
          if (I.lo(k) >= I.hi(k)) continue;
          if (nq[k] > 0 && !(ok = mbar_wait(bar(C::BAR_QFREE + k), (nq[k] - 1) & 1, abort_flag))) break;
          mbar_arrive_expect_tx(bar(C::BAR_Q + k), C::TILE_BYTES);
          for (int c = 0; c < C::NCHUNK; ++c)
            tma_load_4d(sbase + C::OFF_Q + k * C::TILE_BYTES + c * 16384, &tmQ, bar(C::BAR_Q + k), c * 64, I.h,
                        I.row0 + 128 * k, I.b);
          ++nq[k];
        }
        for (int j = I.jb; ok && j < I.je; ++j) {
          for (int kv = 0; kv < 2; ++kv) {
            if (!(ok = mbar_wait(bar(C::BAR_KV_EMPTY + stage), phase ^ 1u, abort_flag))) break;
            mbar_arrive_expect_tx(bar(C::BAR_KV_FULL + stage), C::TILE_BYTES);
            const CUtensorMap* m = kv ? &tmV : &tmK;
            for (int c = 0; c < C::NCHUNK; ++c)
              tma_load_4d(sbase + C::OFF_KV + stage * C::TILE_BYTES + c * 16384, m, bar(C::BAR_KV_FULL + stage),
                          c * 64, hk, 128 * j, I.b);
            ++issued;
            if (++stage == C::NSTAGE) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) break;
        // the next item: take over a CTA of this grid that has not started
        mbar_arrive_expect_tx(bar(C::BAR_CLC), 16);
        clc_try_cancel(resp, bar(C::BAR_CLC));
        clc_pending = true;
        if (!(ok = mbar_wait(bar(C::BAR_CLC), clc_phase, abort_flag))) break;
        clc_pending = false;
        clc_phase ^= 1u;
        item = clc_query(resp);
      }
      if (*abort_flag) {  // let the copies and the cancel request in flight land before the CTA exits
        for (int k = 0; k < 2; ++k)
          if (nq[k] > 0) mbar_wait_drain(bar(C::BAR_Q + k), (nq[k] - 1) & 1);
        for (int i = 0; i < C::NSTAGE && i < issued; ++i) {
          const int n = issued - 1 - i;
          mbar_wait_drain(bar(C::BAR_KV_FULL + n % C::NSTAGE), (n / C::NSTAGE) & 1);
        }
        if (clc_pending) mbar_wait_drain(bar(C::BAR_CLC), clc_phase);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdO = idesc_bf16_f32(128, D, false, true);
      const uint64_t dQ_k = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
      const uint64_t dKV_k = sdesc_sw128(sbase + C::OFF_KV, 16, 1024);
      const uint64_t dKV_mn = sdesc_sw128(sbase + C::OFF_KV, 16384, 1024);
      constexpr uint32_t kTileAdv = C::TILE_BYTES >> 4;
      auto issue_s = [&](int k, int st) {
        const uint64_t a0 = dQ_k + k * kTileAdv;
        const uint64_t b0 = dKV_k + st * kTileAdv;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(tmem + C::TM_S + 128 * k, sdesc_adv(a0, off), sdesc_adv(b0, off), kIdS, kk > 0);
        }
      };
      auto issue_pv = [&](int k, int st, bool first, int kk0) {
        const uint64_t b0 = dKV_mn + st * kTileAdv;
#pragma unroll
        for (int kk = kk0; kk < kk0 + 4; ++kk)
          umma_ts(tmem + C::TM_O + D * k, tmem + C::TM_S + 128 * k + kk * 8, sdesc_adv(b0, kk * 2048), kIdO,
                  (!first || kk > 0));
      };
      int stage = 0;
      uint32_t phase = 0;
      auto take = [&](int& st, uint32_t& ph) {
        st = stage;
        ph = phase;
        if (++stage == C::NSTAGE) {
          stage = 0;
          phase ^= 1u;
        }
      };
      int nq[2] = {0, 0};
      uint32_t pph[2] = {0, 0};
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int slot = n & 1;
        if (!(ok = mbar_wait(bar(C::BAR_ITEM_FULL + slot), (n >> 1) & 1, abort_flag))) break;
        const int item = item_ring[slot];
        mbar_arrive(bar(C::BAR_ITEM_EMPTY + slot));
        if (item < 0) break;
        ModFwdItem I;
        mod_fwd_item(p, item, I);
        // Step j: PV_k(j) and S_k(j + 1) of each query tile whose range holds
        // them; the first step (j = jb - 1) has S products only.  S_k(j + 1)
        // overwrites columns whose P_k(j) was consumed by the PV_k(j) issued
        // just before it.
        for (int j = I.jb - 1; ok && j < I.je; ++j) {
          int vst = -1, nst = -1;
          uint32_t vph = 0, nph = 0;
          if (j >= I.jb) {
            take(vst, vph);
            if (!(ok = mbar_wait(bar(C::BAR_KV_FULL + vst), vph, abort_flag))) break;
          }
          if (j + 1 < I.je) take(nst, nph);
          bool kready = false;
          for (int k = 0; ok && k < 2; ++k) {
            const bool pv = j >= I.lo(k) && j < I.hi(k);
            const bool sn = j + 1 >= I.lo(k) && j + 1 < I.hi(k);
            if (pv) {
              // P arrives in two halves of 64 keys; P_k of the item's first
              // tile also tells that the epilogue of the previous item has
              // read O_k
              if (!(ok = mbar_wait(bar(C::BAR_P + 2 * k), pph[k], abort_flag))) break;
              tc_fence_after();
              issue_pv(k, vst, j == I.lo(k), 0);
              if (!(ok = mbar_wait(bar(C::BAR_P + 2 * k + 1), pph[k], abort_flag))) break;
              pph[k] ^= 1u;
              tc_fence_after();
              issue_pv(k, vst, j == I.lo(k), 4);
            }
            if (sn) {
              if (!kready) {
                if (!(ok = mbar_wait(bar(C::BAR_KV_FULL + nst), nph, abort_flag))) break;
                kready = true;
              }
              if (j + 1 == I.lo(k)) {
                if (!(ok = mbar_wait(bar(C::BAR_Q + k), nq[k] & 1, abort_flag))) break;
                ++nq[k];
              }
              tc_fence_after();
              issue_s(k, nst);
              umma_commit(bar(C::BAR_S + k));
              if (j + 2 == I.hi(k)) umma_commit(bar(C::BAR_QFREE + k));  // Q_k read for the last time
            } else if (pv) {
              umma_commit(bar(C::BAR_OFIN + k));  // PV of the range's last tile: O_k final
            }
          }
          if (!ok) break;
          if (vst >= 0) umma_commit(bar(C::BAR_KV_EMPTY + vst));
          if (nst >= 0) {
            // a stage is handed back only after its load has landed, used or not
            if (!kready && !(ok = mbar_wait(bar(C::BAR_KV_FULL + nst), nph, abort_flag))) break;
            umma_commit(bar(C::BAR_KV_EMPTY + nst));
          }
        }
      }
      if (*abort_flag) {  // wait for every MMA this thread issued before tensor memory is freed
        umma_commit(bar(C::BAR_DRAIN));
        mbar_wait_drain(bar(C::BAR_DRAIN), 0);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax / epilogue
    regs_set<200, kLaunchRegs>();
    const int k = warp >> 2;
    const int t = threadIdx.x & 127;
    const int wq = warp & 3;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tS = lane_base + C::TM_S + 128 * k;
    const uint32_t tO = lane_base + C::TM_O + D * k;
    const uint32_t ost = sbase + C::OFF_OST + k * C::OST_BYTES + wq * 4096;
    uint32_t sph = 0;
    uint32_t oph = 0;
    for (int n = 0;; ++n) {
      const int slot = n & 1;
      bool ok = mbar_wait(bar(C::BAR_ITEM_FULL + slot), (n >> 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int item = item_ring[slot];
      mbar_arrive(bar(C::BAR_ITEM_EMPTY + slot));
      if (item < 0) break;
      ModFwdItem I;
      mod_fwd_item(p, item, I);
      const int qi = I.row0 + 128 * k + t;  // this thread's query
      int2 see = make_int2(0, 0);
      if (qi < p.N) see = p.plan.rows[static_cast<size_t>(I.b) * p.N + qi];
      float slope = 0.f;
      if (BIAS) slope = slope_log2(p.slopes[I.h]);
      // no key after the query is visible: the bias is one-sided on every tile
      const bool behind = see.y <= qi + 1;
      float m = -INFINITY;         // reference max, log2 units
      uint64_t lsum[2] = {0, 0};   // unrounded P, packed pairs
      uint64_t rsum[2] = {0, 0};   // bf16-rounded P, packed pairs
      for (int j = I.lo(k); j < I.hi(k); ++j) {
        ok = mbar_wait(bar(C::BAR_S + k), sph, abort_flag);
        sph ^= 1u;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + 32 * cc, s[cc]);
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) tmem_wait_ld(s[cc]);
        const int kbase = 128 * j;
        // ---- scores to base-2 logits z, in place.  Without cap and bias s
        // stays raw and the scale is applied with the exponent below.
        if constexpr (CAP || BIAS) {
          float side_slope = 0.f;  // -slope below the diagonal, +slope above it: times i - j
          bool straddle = false;
          if constexpr (BIAS) {
            const bool below = behind || kbase + 127 <= qi;
            const bool above = kbase >= qi;
            const bool all_below = __all_sync(0xffffffffu, below), all_above = __all_sync(0xffffffffu, above);
            straddle = !(all_below || all_above);
            side_slope = straddle ? 0.f : (all_below ? -slope : slope);
          }
          const float dist0 = static_cast<float>(qi - kbase);
          uint64_t d2 = f2_pack(dist0, dist0 - 1.f);
          const uint64_t m2 = f2_pack(-2.f, -2.f), ss2 = f2_pack(side_slope, side_slope);
          if constexpr (CAP) {
            float ax = 0.f;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc)
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                ax = fmax3(ax, fabsf(__uint_as_float(s[cc][i])), fabsf(__uint_as_float(s[cc][i + 1])));
            const uint64_t xm2 = f2_pack(p.x_mul, p.x_mul), cl2 = f2_pack(p.cap_log2, p.cap_log2);
            if (__all_sync(0xffffffffu, ax * fabsf(p.x_mul) <= kTanhRange)) {
#pragma unroll
              for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const uint64_t x = fmul2(f2_pack(__uint_as_float(s[cc][i]), __uint_as_float(s[cc][i + 1])), xm2);
                  const uint64_t th = tanh2_poly(x);
                  uint64_t z = fmul2(th, cl2);
                  if constexpr (BIAS) {
                    z = ffma2(ss2, d2, z);
                    d2 = fadd2(d2, m2);
                  }
                  float z0, z1;
                  f2_unpack(z, z0, z1);
                  s[cc][i] = __float_as_uint(z0);
                  s[cc][i + 1] = __float_as_uint(z1);
                }
            } else {
              const float xe = p.x_mul * kTwoLog2e;
              const uint64_t xe2 = f2_pack(xe, xe), cm2 = f2_pack(-2.f * p.cap_log2, -2.f * p.cap_log2);
#pragma unroll
              for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  uint64_t z = tanh2_any(fmul2(f2_pack(__uint_as_float(s[cc][i]), __uint_as_float(s[cc][i + 1])), xe2),
                                         cl2, cm2);
                  if constexpr (BIAS) {
                    z = ffma2(ss2, d2, z);
                    d2 = fadd2(d2, m2);
                  }
                  float z0, z1;
                  f2_unpack(z, z0, z1);
                  s[cc][i] = __float_as_uint(z0);
                  s[cc][i + 1] = __float_as_uint(z1);
                }
            }
          } else {
            const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
#pragma unroll
            for (int cc = 0; cc < 4; ++cc)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float z0, z1;
                const uint64_t y = fmul2(f2_pack(__uint_as_float(s[cc][i]), __uint_as_float(s[cc][i + 1])), c2);
                f2_unpack(ffma2(ss2, d2, y), z0, z1);
                d2 = fadd2(d2, m2);
                s[cc][i] = __float_as_uint(z0);
                s[cc][i + 1] = __float_as_uint(z1);
              }
          }
          if constexpr (BIAS) {
            if (straddle) {
              float dist = dist0;
#pragma unroll
              for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  s[cc][i] = __float_as_uint(fmaf(-slope, fabsf(dist), __uint_as_float(s[cc][i])));
                  dist -= 1.f;
                }
            }
          }
        }
        // ---- mask: keys outside [see.x, see.y)
        if (kbase < see.x || kbase + 128 > see.y) {
          const int lo = see.x - kbase, hi = see.y - kbase;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            // bits [lo, hi) of the chunk's 32 columns
            const int l32 = min(max(lo - 32 * cc, 0), 32), h32 = min(max(hi - 32 * cc, 0), 32);
            const uint32_t seen = (h32 == 32 ? 0xffffffffu : (1u << h32) - 1u) & (l32 == 32 ? 0u : 0xffffffffu << l32);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen & (1u << i))) s[cc][i] = __float_as_uint(-INFINITY);
          }
        }
        // ---- row max: four independent chains of three-input maxima
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
#pragma unroll
          for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int a = 0; a < 4; ++a)
              mx[a] = fmax3(mx[a], __uint_as_float(s[cc][i + 2 * a]), __uint_as_float(s[cc][i + 2 * a + 1]));
        const float mraw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float mt = (CAP || BIAS) ? mraw : mraw * p.scale_log2;
        const bool move = (mt > m + kRescaleThreshold) || (m == -INFINITY && mt > -INFINITY);
        float alpha = 1.f;
        if (move) {
          alpha = ex2(m - mt);  // 0 when m was -inf
          m = mt;
        }
        if (__any_sync(0xffffffffu, move)) {  // warp-uniform: tcgen05 loads and stores below
          const uint64_t a2 = f2_pack(alpha, alpha);
          lsum[0] = fmul2(lsum[0], a2);
          lsum[1] = fmul2(lsum[1], a2);
          rsum[0] = fmul2(rsum[0], a2);
          rsum[1] = fmul2(rsum[1], a2);
          if (j > I.lo(k)) {
            // rescale this row of the partial output; PV(j-1) has completed
            // because the commit that signalled S(j) was issued after it
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * q, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + 32 * q, o);
            }
            tmem_wait_st();
          }
        }
        const float neg_m = (m == -INFINITY) ? 0.f : -m;
        const uint64_t nm2 = f2_pack(neg_m, neg_m);
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t z = f2_pack(__uint_as_float(s[cc][2 * i]), __uint_as_float(s[cc][2 * i + 1]));
            float x0, x1;
            f2_unpack((CAP || BIAS) ? fadd2(z, nm2) : ffma2(z, c2, nm2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            const uint32_t w = pack_bf16x2(p0, p1);
            pk[i] = w;
            lsum[i & 1] = fadd2(lsum[i & 1], f2_pack(p0, p1));
            rsum[i & 1] = fadd2(rsum[i & 1], f2_pack(bf16lo_to_f32(w), bf16hi_to_f32(w)));
          }
          tmem_st16(tS + 16 * cc, pk);
          if (cc == 1) {  // first 64 keys of P are in place
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(C::BAR_P + 2 * k));
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::BAR_P + 2 * k + 1));
      }
      if (!ok) break;
      // ---- epilogue: O / l~ through this warp's staging rows, LSE.  A tile
      // that meets no key has no product to wait for: its rows are zero.
      const bool any = I.lo(k) < I.hi(k);
      if (any) {
        ok = mbar_wait(bar(C::BAR_OFIN + k), oph, abort_flag);
        oph ^= 1u;
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
      }
      const float l = f2_sum(lsum[0]) + f2_sum(lsum[1]);
      const float r = f2_sum(rsum[0]) + f2_sum(rsum[1]);
      // an exact zero: a row that saw nothing (else the key that set the reference
      // maximum has added 1 since the sums were last rescaled; NaN scores give NaN
      // sums and stay NaN)
      const bool empty = l == 0.f;
      const float inv = empty ? 0.f : 1.f / r;
      const uint64_t inv2 = f2_pack(inv, inv);
      const int wrow = I.row0 + 128 * k + 32 * wq;  // this warp's first row
      const size_t grow0 = static_cast<size_t>(I.b) * p.N + wrow;
      const int rows_left = p.N - wrow;
      if (rows_left > 0) {
#pragma unroll 1
        for (int hf = 0; hf < D / 64; ++hf) {
          uint32_t o[2][32];
          // loaded even where the tile met no key: a load under a condition would
          // keep these registers live through the tile loop
          tmem_ld32(tO + 64 * hf, o[0]);
          tmem_ld32(tO + 64 * hf + 32, o[1]);
          tmem_wait_ld(o[0]);
          tmem_wait_ld(o[1]);
          uint32_t low[32];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t w[4];
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                float a, b2;
                f2_unpack(fmul2(f2_pack(__uint_as_float(o[e][8 * u + 2 * v]), __uint_as_float(o[e][8 * u + 2 * v + 1])),
                                inv2),
                          a, b2);
                if (empty) a = b2 = 0.f;  // its accumulator columns may hold anything
                w[v] = pack_bf16x2(a, b2);
                low[16 * e + 4 * u + v] = pack_bf16x2(a - bf16lo_to_f32(w[v]), b2 - bf16hi_to_f32(w[v]));
              }
              st_shared_v4(ost + sw128_offset(lane, 4 * e + u), w[0], w[1], w[2], w[3]);
            }
          for (int part = 0; part < (p.o_low ? 2 : 1); ++part) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(part ? p.o_low : p.o);
            if (part) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                st_shared_v4(ost + sw128_offset(lane, q), low[4 * q], low[4 * q + 1], low[4 * q + 2], low[4 * q + 3]);
            }
            __syncwarp();
            // read back 4 rows x 128 bytes per instruction: coalesced 16-byte stores
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int e = 32 * i + lane;
              const int rr = e >> 3, q = e & 7;
              uint32_t a0, a1, a2, a3;
              ld_shared_v4(ost + sw128_offset(rr, q), a0, a1, a2, a3);
              if (rr < rows_left)
                st_global_v4(dst + ((grow0 + rr) * p.H + I.h) * D + 64 * hf + 8 * q, a0, a1, a2, a3);
            }
            __syncwarp();
          }
        }
        if (qi < p.N)
          p.lse[(static_cast<size_t>(I.b) * p.H + I.h) * p.N + qi] = empty ? -INFINITY : (m + lg2(l)) * kLn2;
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
