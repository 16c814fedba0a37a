// Modified-score attention, backward, for sm_100a.  With the notation of
// fa_mod_fwd.cuh and t_ij = tanh(x_ij / cap):
//
//     P_ij  = exp(z_ij - LSE_i)                   recomputed, 0 outside the mask
//     D_i   = sum_c dO_ic O_ic
//     dP    = dO V^T
//     dS_ij = P_ij (1 - t_ij^2) (dP_ij - D_i)     (the factor only with CAP)
//     dV_j  = sum P_ij dO_i        over the queries and the heads of the group
//     dK_j  = scale sum dS_ij q_i  likewise
//     dQ_i  = scale sum dS_ij k_j
//
// Three launches, as in the plain backward (fa_bwd.cuh): D and the zeroed fp32
// dQ accumulator; the fused main kernel; dQ to bf16.  The second and third are
// launched as dependents of the one before (2 x 8(1) x 2047 x 64, window: 66 us
// with four plain launches, 63 so; 1 x 2(1) x 130 x 64: 25 and 22).  The main kernel is the
// plain one's pipeline (same warps, barriers, tensor-memory columns and
// products, S^T form with one key per lane) with these differences:
//   - a work item is (128-key tile, batch entry, key head); the CTA walks the
//     query tiles of the mask plan's range for that key tile, for every query
//     head of the group in turn, so dK and dV of a shared key head accumulate
//     in tensor memory over the whole group: no atomics, no second pass, a
//     fixed order.  A key tile no query sees is stored as zero.  Where that
//     makes too few items for the SMs (few key heads, short sequences) the host
//     splits each group's heads over several items; those store fp32 partial
//     sums, and the last kernel adds them in a fixed order: 2 x 8 heads on one key
//     head x 2047 tokens, window 512, takes 32 items whole (181 us) and 256
//     split;
//   - D takes O with its rounding residual when the caller has it: with O in
//     bf16 alone, rows that one key dominates (P near 1, dP - D near 0) lose
//     bits: relative error of dQ 5.2e-3 against 3.0e-3 at q = 8 N(0,1),
//     k = N(0,1), d = 64, N = 1024;
//   - the row term of the exponent, -LSE_i log2 e, carries the query's part of
//     a one-sided distance bias (the key's part is one constant per thread), for
//     slopes up to 4: see kSplitSlope;
//   - between its two phases the thread keeps P (1 - t^2) 2^15 in fp16 for dS:
//     one register per pair as with bf16(P), but with an error of 2^-11 instead
//     of 2^-8 down to P = 2^-29 (below, 2^-40 absolute: less than the rounding
//     of any row's larger terms), which leaves the rounding of dS to bf16 as the
//     one that shows (relative error of dQ 2.4e-3, with bf16 there 3.0e-3).
//
// Bound like the plain backward (shared-memory operands, the P and dS chain):
// ncu sees 35% of the tensor pipe and 38% of the issue slots busy with the cap.
// At 4 x 16(4) x 4096 x 128 causal (687 GFLOP) the call takes 0.99-1.10 ms with a cap
// and 0.89-0.99 without; with 16 key heads 1.04-1.20 and 0.94-1.10, where the plain
// backward takes 0.89-0.97 in the same runs (the low ends one call at a time, the
// high ends back to back under the power cap).
#pragma once
#include <cuda_fp16.h>

#include <type_traits>

#include "fa_bwd.cuh"
#include "fa_mod_fwd.cuh"

namespace fa {

// Steepest bias whose two parts, the query's and the key's, are rounded apart: both
// reach 127 slope log2(e) where the distance may be 0, and four roundings of that size
// put an error of at most 3.1e-5 slope (relative) into P: here 1.2e-4, a quarter of
// the rounding of P to fp16.  Steeper ones take the exact distance element by element
// (that of 3000 would lose 2% of the diagonal's P, that of 1e5 overflow it), at
// 2 x 16 x 8192 x 64 with documents in 466 us where two parts take 441.
constexpr float kSplitSlope = 4.f;
constexpr float kDsUp = 32768.f;  // P <= 1 (and a rounding) times this stays finite in fp16

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct ModBwdParams {
  const void* o;
  const void* o_low;    // bf16 residual of O, or nullptr
  const void* dout;
  const float* lse;
  const float* slopes;  // [H], BIAS
  void* dk;
  void* dv;
  float* dk_part;       // fp32 [B, N, Hv, d] partial dK (unscaled) and dV when a
  float* dv_part;       // group's heads are split, else nullptr
  float* dq_acc;        // layout: dq_acc_index4(); nullptr: dQ has a pass of its own
  void* dq;             // written by that pass or the conversion
  float* dvec;          // fp32 D [B, H, N]
  PlanView plan;
  int B, N, H, Hkv, G;
  int Hv, hs;           // items of a key tile in a batch entry, hs = H / Hv query heads each
  int T;                // ceil(N / 128)
  int group;            // (entry, heads) pairs per scheduling group
  float scale, scale_log2, x_mul, cap_log2;
};

// 32 scores of a thread (raw products) become tanh(x / cap); the whole warp calls
__device__ __forceinline__ void cap_scores(uint32_t (&s)[32], float x_mul) {
  float ax = 0.f;
#pragma unroll
  for (int e = 0; e < 32; e += 2) ax = fmax3(ax, fabsf(__uint_as_float(s[e])), fabsf(__uint_as_float(s[e + 1])));
  if (__all_sync(0xffffffffu, ax * fabsf(x_mul) <= kTanhRange)) {
    const uint64_t xm2 = f2_pack(x_mul, x_mul);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float a, b;
      f2_unpack(tanh2_poly(fmul2(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), xm2)), a, b);
      s[e] = __float_as_uint(a);
      s[e + 1] = __float_as_uint(b);
    }
  } else {
    const uint64_t xe2 = f2_pack(x_mul * kTwoLog2e, x_mul * kTwoLog2e);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float a, b;
      f2_unpack(tanh2_any(fmul2(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), xe2), f2_pack(1.f, 1.f),
                          f2_pack(-2.f, -2.f)), a, b);
      s[e] = __float_as_uint(a);
      s[e + 1] = __float_as_uint(b);
    }
  }
}

// D = rowsum(dO (O + O_low)) and the zeroed dQ accumulator; the shape of
// fa_bwd_preprocess_kernel.
template <int D>
__global__ void __launch_bounds__(256) fa_mod_bwd_preprocess_kernel(const ModBwdParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPW = 32 / LPR;
  const int64_t nthreads = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t gtid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t nrows = static_cast<int64_t>(p.B) * p.N * p.H;
  const int64_t nacc4 = nrows * (D / 4);
  float4* acc = reinterpret_cast<float4*>(p.dq_acc);
  if (acc)
    for (int64_t i = gtid; i < nacc4; i += nthreads) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, part = lane % LPR;
  const int64_t nwarps = nthreads >> 5;
  constexpr int U = 4;  // warp steps whose loads are in flight together
  for (int64_t w0 = (gtid >> 5) * U; w0 * RPW < nrows; w0 += nwarps * U) {
    uint4 ov[U], gv[U], lv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = (w0 + u) * RPW + sub;
      ov[u] = gv[u] = lv[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row < nrows) {
        const size_t off = static_cast<size_t>(row) * D + part * 8;
        ov[u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.o) + off);
        gv[u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.dout) + off);
        if (p.o_low) lv[u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.o_low) + off);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = (w0 + u) * RPW + sub;
      const uint32_t ow[4] = {ov[u].x, ov[u].y, ov[u].z, ov[u].w}, gw[4] = {gv[u].x, gv[u].y, gv[u].z, gv[u].w},
                     lw[4] = {lv[u].x, lv[u].y, lv[u].z, lv[u].w};
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum = fmaf(bf16lo_to_f32(ow[e]) + bf16lo_to_f32(lw[e]), bf16lo_to_f32(gw[e]), sum);
        sum = fmaf(bf16hi_to_f32(ow[e]) + bf16hi_to_f32(lw[e]), bf16hi_to_f32(gw[e]), sum);
      }
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (part == 0 && row < nrows) {
        const int64_t tok = row / p.H;
        const int h = static_cast<int>(row % p.H);
        const int64_t b = tok / p.N, n = tok % p.N;
        p.dvec[(static_cast<size_t>(b) * p.H + h) * p.N + n] = sum;
      }
    }
  }
}

template <int D>
struct ModBwdCfg : BwdCfg<D> {
  using Base = BwdCfg<D>;
  // visible key range of each query column, relative to the key tile:
  // 128 words lo | len << 16 behind the D vector
  static constexpr int OFF_SEE = Base::OFF_BAR;
  static constexpr int OFF_BAR = OFF_SEE + 512;
  static constexpr int OFF_MISC = (OFF_BAR + Base::NBAR * 8 + 15) & ~15;
  static constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// One work item: (128-key tile j, batch entry, heads of a key head).  They go in
// groups of p.group (entry, heads) pairs, inside a group early key tiles first:
// under a causal mask they meet the most query tiles, and the longest items have
// to start first for the persistent CTAs to end together.  The host makes the
// whole batch one group up to 4096 items; with more, the end of the launch
// weighs little and groups whose Q, dO and dQ rows stay in L2 are faster.
// Measured, one group against L2-sized ones: 4 x 16(4) x 4096 x 128 (512 items)
// 1069 us, 1407; 1 x 8(2) x 16384 x 128 (1024) 1911, 2497; 1 x 16 x 16384 x 128
// (2048) 3375, 3466; 16 x 32 x 2048 x 64 (8192) 1735, 1565.
struct ModBwdItem {
  int hv, hk, b, k0, i_begin, ni, niter;  // niter = ni query tiles x hs heads
};

__device__ __forceinline__ void mod_bwd_item(const ModBwdParams& p, int c, ModBwdItem& it) {
  const int nbh = p.B * p.Hv;
  const int g = c / (p.group * p.T);
  const int gs = min(p.group, nbh - g * p.group);
  const int cidx = c - g * p.group * p.T;
  const int bh = g * p.group + cidx % gs;
  const int j = cidx / gs;
  it.hv = bh % p.Hv;
  it.hk = it.hv * p.hs / p.G;
  it.b = bh / p.Hv;
  it.k0 = 128 * j;
  const PlanKTile kt = p.plan.kt[static_cast<size_t>(it.b) * p.T + j];
  it.i_begin = max(kt.qbeg, 0);  // clamped as in the forward pass
  it.ni = max(min(kt.qend, p.T) - it.i_begin, 0);
  it.niter = it.ni * p.hs;
}

// DQ: also form dQ_i = dS K_j per tile and add it into the fp32 accumulator
// (atomic, order varies); without it the kernel computes dK and dV only and
// fa_mod_bwd_dq.cuh sums dQ in a fixed order.
template <int D, bool CAP, bool BIAS, bool DQ>
__global__ void __launch_bounds__(512, 1)
    fa_mod_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                  const ModBwdParams p) {
  using C = ModBwdCfg<D>;
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
    mbar_init(bar(C::BAR_KV), 1);
    for (int s = 0; s < C::NSTAGE; ++s) {
      mbar_init(bar(C::BAR_QDO_FULL + s), 1);
      mbar_init(bar(C::BAR_QDO_EMPTY + s), 1);
    }
    mbar_init(bar(C::BAR_S), 1);
    mbar_init(bar(C::BAR_DP), 1);
    mbar_init(bar(C::BAR_P), 256);
    mbar_init(bar(C::BAR_DS), 256);
    mbar_init(bar(C::BAR_DS_EMPTY), 1);
    mbar_init(bar(C::BAR_DQ_FULL), 1);
    mbar_init(bar(C::BAR_DQ_EMPTY), 128);
    mbar_init(bar(C::BAR_ACC), 1);
    mbar_init(bar(C::BAR_DRAIN), 1);
    mbar_init(bar(C::BAR_KV_EMPTY), 1);
    mbar_init(bar(C::BAR_ACC_FREE), 256);
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar(C::BAR_ITEM_FULL + k), 1);
      mbar_init(bar(C::BAR_ITEM_EMPTY + k), C::ITEM_CONSUMERS);
    }
    mbar_init(bar(C::BAR_CLC), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  // D and the zeroed accumulator are there.  No memory clobber: the barrier below
  // keeps every access after this, and with one the bias variants spill 40 bytes
  // instead of 16.  The kernel before this one does not call for its dependents
  // early: CTAs placed while it still runs took the long first items unevenly
  // (2 x 16 x 8192 x 64 with documents: 281 us against 273).
  asm volatile("griddepcontrol.wait;" ::);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Item n of this CTA from the two-slot ring the producer fills; -1 ends.
  auto take_item = [&](int n, bool& ok) -> int {
    const int slot = n & 1;
    ok = mbar_wait(bar(C::BAR_ITEM_FULL + slot), (n >> 1) & 1, abort_flag);
    if (!ok) return -1;
    const int item = item_ring[slot];
    mbar_arrive(bar(C::BAR_ITEM_EMPTY + slot));
    return item;
  };
  if (warp >= 12) {
    regs_set<C::REGS_PRODUCER, C::LAUNCH_REGS>();
  }
  if (warp == 12) {
    // ------------------------------------------------------------ producer and scheduler
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmdO);
      int item = blockIdx.x;
      int nitems = 0;  // items whose K, V were loaded
      int gt = 0;      // Q/dO tiles loaded (all items)
      uint32_t clc_phase = 0;
      bool clc_pending = false;
      bool ok = true;
      for (int n = 0; ok;) {
        const int slot = n & 1;
        if (n >= 2 && !(ok = mbar_wait(bar(C::BAR_ITEM_EMPTY + slot), ((n >> 1) - 1) & 1, abort_flag))) break;
        item_ring[slot] = item;
        mbar_arrive(bar(C::BAR_ITEM_FULL + slot));
        ++n;
        if (item < 0) break;
        ModBwdItem I;
        mod_bwd_item(p, item, I);
        // ask for the next item now; the answer is read once this item's loads are issued
        mbar_arrive_expect_tx(bar(C::BAR_CLC), 16);
        clc_try_cancel(resp, bar(C::BAR_CLC));
        clc_pending = true;
        if (I.niter > 0) {
          // K_j, V_j replace the previous item's once its products are done
          if (nitems > 0 && !(ok = mbar_wait(bar(C::BAR_KV_EMPTY), (nitems - 1) & 1, abort_flag))) break;
          mbar_arrive_expect_tx(bar(C::BAR_KV), 2 * C::TILE_BYTES);
          for (int c = 0; c < C::NCHUNK; ++c) {
            tma_load_4d(sbase + C::OFF_K + c * 16384, &tmK, bar(C::BAR_KV), c * 64, I.hk, I.k0, I.b);
            tma_load_4d(sbase + C::OFF_V + c * 16384, &tmV, bar(C::BAR_KV), c * 64, I.hk, I.k0, I.b);
          }
          ++nitems;
          int h = I.hv * p.hs, i = 0;  // query head and tile of the walk
          for (int it = 0; it < I.niter; ++it, ++gt) {
            const int st = gt % C::NSTAGE;
            const uint32_t ph = (gt / C::NSTAGE) & 1;
            if (!(ok = mbar_wait(bar(C::BAR_QDO_EMPTY + st), ph ^ 1u, abort_flag))) break;
            const int q0 = 128 * (I.i_begin + i);
            mbar_arrive_expect_tx(bar(C::BAR_QDO_FULL + st), 2 * C::TILE_BYTES);
            for (int c = 0; c < C::NCHUNK; ++c) {
              tma_load_4d(sbase + C::OFF_Q + st * C::TILE_BYTES + c * 16384, &tmQ, bar(C::BAR_QDO_FULL + st), c * 64,
                          h, q0, I.b);
              tma_load_4d(sbase + C::OFF_DO + st * C::TILE_BYTES + c * 16384, &tmdO, bar(C::BAR_QDO_FULL + st),
                          c * 64, h, q0, I.b);
            }
            if (++i == I.ni) {
              i = 0;
              ++h;
            }
          }
          if (!ok) break;
        }
        if (!(ok = mbar_wait(bar(C::BAR_CLC), clc_phase, abort_flag))) break;
        clc_pending = false;
        clc_phase ^= 1u;
        item = clc_query(resp);
      }
      if (*abort_flag) {  // let the copies and the cancel request in flight land before the CTA exits
        if (nitems > 0) mbar_wait_drain(bar(C::BAR_KV), (nitems - 1) & 1);
        for (int i = 0; i < C::NSTAGE && i < gt; ++i) {
          const int n = gt - 1 - i;
          mbar_wait_drain(bar(C::BAR_QDO_FULL + n % C::NSTAGE), (n / C::NSTAGE) & 1);
        }
        if (clc_pending) mbar_wait_drain(bar(C::BAR_CLC), clc_phase);
      }
    }
    __syncwarp();
  } else if (warp == 13) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdSq = idesc_bf16_f32(128, 128, false, false);  // S^T, dP^T
      constexpr uint32_t kIdDV = idesc_bf16_f32(128, D, false, true);     // dV (A in TMEM), dK
      constexpr uint32_t kIdDQ = idesc_bf16_f32(128, D, true, true);      // dQ: A = dS (MN-major view)
      // operand descriptors, built once; per MMA only the start address moves
      const uint64_t dK_k = sdesc_sw128(sbase + C::OFF_K, 16, 1024);        // K as K-major A of S^T
      const uint64_t dV_k = sdesc_sw128(sbase + C::OFF_V, 16, 1024);        // V as K-major A of dP^T
      const uint64_t dK_mn = sdesc_sw128(sbase + C::OFF_K, 16384, 1024);    // K as MN-major B of dQ
      const uint64_t dS_k = sdesc_sw128(sbase + C::OFF_DS, 16, 1024);       // dS^T as K-major A of dK
      const uint64_t dS_mn = sdesc_sw128(sbase + C::OFF_DS, 16384, 1024);   // dS as MN-major A of dQ
      const uint64_t dQ0_k = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);       // Q stage 0, K-major B of S^T
      const uint64_t dQ0_mn = sdesc_sw128(sbase + C::OFF_Q, 16384, 1024);   // Q stage 0, MN-major B of dK
      const uint64_t dO0_k = sdesc_sw128(sbase + C::OFF_DO, 16, 1024);      // dO stage 0, K-major B of dP^T
      const uint64_t dO0_mn = sdesc_sw128(sbase + C::OFF_DO, 16384, 1024);  // dO stage 0, MN-major B of dV
      constexpr uint32_t kStageAdv = C::TILE_BYTES >> 4;
      auto issue_s = [&](int gt) {  // S^T = K Q_gt^T
        const uint64_t bq = dQ0_k + (gt % C::NSTAGE) * kStageAdv;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(tmem + C::TM_S, sdesc_adv(dK_k, off), sdesc_adv(bq, off), kIdSq, kk > 0);
        }
        umma_commit(bar(C::BAR_S));
      };
      auto issue_dp = [&](int gt) {  // dP^T = V dO_gt^T
        const uint64_t bo = dO0_k + (gt % C::NSTAGE) * kStageAdv;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_ss(tmem + C::TM_DP, sdesc_adv(dV_k, off), sdesc_adv(bo, off), kIdSq, kk > 0);
        }
        umma_commit(bar(C::BAR_DP));
      };
      // Order per query tile i:  dV(i)  S^T(i+1)  dK(i)  dQ(i)  dP^T(i+1).
      // dP^T does not depend on P, so dP^T(i+1) is issued as soon as its
      // columns are free (the P/dS warps have read dP^T(i) and, at d = 128,
      // the drain has emptied dQ(i), which shares them): the P/dS warps then
      // go from P^T(i+1) straight on to dS^T(i+1), and P^T(i+1) is computed
      // while dK(i) and dQ(i) run.
      int gt0 = 0;     // tiles of earlier items
      int nitems = 0;  // items done
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int item = take_item(n, ok);
        if (!ok || item < 0) break;
        ModBwdItem I;
        mod_bwd_item(p, item, I);
        const int niter = I.niter;
        if (niter == 0) continue;
        if (!(ok = mbar_wait(bar(C::BAR_KV), nitems & 1, abort_flag))) break;
        if (!(ok = mbar_wait(bar(C::BAR_QDO_FULL + gt0 % C::NSTAGE), (gt0 / C::NSTAGE) & 1, abort_flag))) break;
        tc_fence_after();
        issue_s(gt0);
        // at d = 128 the first dP^T reuses the columns of the previous item's last dQ
        if (DQ && C::DQ_ALIASES_DP && gt0 > 0) {
          if (!(ok = mbar_wait(bar(C::BAR_DQ_EMPTY), (gt0 - 1) & 1, abort_flag))) break;
          tc_fence_after();
        }
        issue_dp(gt0);
        for (int it = 0; ok && it < niter; ++it) {
          const int gt = gt0 + it;
          const int st = gt % C::NSTAGE;
          const uint32_t par = gt & 1;
          const uint64_t q_mn = dQ0_mn + st * kStageAdv;
          const uint64_t o_mn = dO0_mn + st * kStageAdv;
          // dV += P^T dO   (A = P^T packed bf16 in tensor memory)
          if (!(ok = mbar_wait(bar(C::BAR_P), par, abort_flag))) break;
          if (it == 0 && nitems > 0) {  // the previous item's dK, dV have been read out
            if (!(ok = mbar_wait(bar(C::BAR_ACC_FREE), (nitems - 1) & 1, abort_flag))) break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            // queries 16kk..16kk+15 of P^T: columns 8kk (first 64 queries) or 32 + 8kk (last 64)
            umma_ts(tmem + C::TM_DV, tmem + C::TM_S + kk * 8 + (kk >= 4 ? 32 : 0), sdesc_adv(o_mn, kk * 2048), kIdDV,
                    (it > 0 || kk > 0));
          // S^T of the next query tile (P^T(i) was consumed by dV above, in issue order)
          if (it + 1 < niter) {
            const int st1 = (gt + 1) % C::NSTAGE;
            if (!(ok = mbar_wait(bar(C::BAR_QDO_FULL + st1), ((gt + 1) / C::NSTAGE) & 1, abort_flag))) break;
            tc_fence_after();
            issue_s(gt + 1);
          }
          // dK += dS^T Q ;  dQ_i = dS K
          if (!(ok = mbar_wait(bar(C::BAR_DS), par, abort_flag))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ss(tmem + C::TM_DK, sdesc_adv(dS_k, (kk >> 2) * 16384 + (kk & 3) * 32), sdesc_adv(q_mn, kk * 2048),
                    kIdDV, (it > 0 || kk > 0));
          if constexpr (DQ) {
            if (!C::DQ_ALIASES_DP && gt > 0) {
              if (!(ok = mbar_wait(bar(C::BAR_DQ_EMPTY), par ^ 1u, abort_flag))) break;
              tc_fence_after();
            }
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ss(tmem + C::TM_DQ, sdesc_adv(dS_mn, kk * 2048), sdesc_adv(dK_mn, kk * 2048), kIdDQ, kk > 0);
          }
          umma_commit(bar(C::BAR_QDO_EMPTY + st));
          umma_commit(bar(C::BAR_DS_EMPTY));
          if (DQ) umma_commit(bar(C::BAR_DQ_FULL));
          // dP^T of the next query tile: the P/dS warps finished reading dP^T(i)
          // before they signalled dS^T(i); at d = 128 its columns also hold dQ(i),
          // so wait until the drain has loaded it (completion i of DQ_EMPTY)
          if (it + 1 < niter) {
            if (DQ && C::DQ_ALIASES_DP) {
              if (!(ok = mbar_wait(bar(C::BAR_DQ_EMPTY), par, abort_flag))) break;
              tc_fence_after();
            }
            issue_dp(gt + 1);
          }
        }
        if (!ok) break;
        umma_commit(bar(C::BAR_ACC));       // dK, dV of this item complete
        umma_commit(bar(C::BAR_KV_EMPTY));  // and no product reads K, V any more
        gt0 += niter;
        ++nitems;
      }
      if (*abort_flag) {
        umma_commit(bar(C::BAR_DRAIN));
        mbar_wait_drain(bar(C::BAR_DRAIN), 0);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ P^T and dS^T
    regs_set<C::REGS_PDS, C::LAUNCH_REGS>();
    const int w = warp >> 2;          // this warpgroup's query columns: 64w .. 64w+63
    const int t = threadIdx.x & 127;  // key row within the tile == tensor-memory lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* sLSE = reinterpret_cast<float*>(smem + C::OFF_LSE);
    float* sDv = reinterpret_cast<float*>(smem + C::OFF_DV);
    uint32_t* sSee = reinterpret_cast<uint32_t*>(smem + C::OFF_SEE);
    constexpr float kLog2e = 1.4426950408889634f;
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
    int gt0 = 0;
    int nitems = 0;
    for (int n = 0;; ++n) {
      bool ok;
      const int item = take_item(n, ok);
      if (!__all_sync(0xffffffffu, ok) || item < 0) break;
      ModBwdItem I;
      mod_bwd_item(p, item, I);
      const int k0 = I.k0;
      const int key = k0 + t;
      const bool key_ok = key < p.N;
      // The terms of this warpgroup's query columns, thread t < 64 those of
      // column 64w + t of a tile: LSE, D, the keys that the query sees; and the
      // tile's own.  They are loaded a tile ahead and only touched when that
      // tile starts: any arithmetic on them here would wait for the loads.
      float n_lse, n_dv, n_slope = 0.f;
      int2 n_see;
      int n_lo, n_hi, n_ahead;
      auto fetch = [&](int h, int q0) {
        const PlanQTile* qt = p.plan.qt + static_cast<size_t>(I.b) * p.T + (q0 >> 7);
        n_lo = qt->full_lo;
        n_hi = qt->full_hi;
        if constexpr (BIAS) {
          n_ahead = qt->ahead;
          n_slope = p.slopes[h];
        }
        const int q = q0 + 64 * w + t;
        if (t < 64 && q < p.N) {
          const size_t li = (static_cast<size_t>(I.b) * p.H + h) * p.N + q;
          n_lse = p.lse[li];
          n_dv = p.dvec[li];
          n_see = p.plan.rows[static_cast<size_t>(I.b) * p.N + q];
        } else {  // a row past the end: -LSE = -inf, so P is exactly 0
          n_lse = INFINITY;
          n_dv = 0.f;
          n_see = make_int2(0, 0);
        }
      };
      int h = I.hv * p.hs, i = 0;
      if (I.niter > 0) fetch(h, 128 * I.i_begin);
      for (int it = 0; it < I.niter; ++it) {
        const uint32_t par = (gt0 + it) & 1;
        const int q0 = 128 * (I.i_begin + i);
        named_bar_sync(1 + w, 128);  // the warpgroup is done with the previous tile's values
        const bool tile_full = k0 >= n_lo && k0 + 128 <= n_hi;
        // How the bias runs over the tile pair: below the diagonal (or no row
        // sees past itself) +1, above it -1, both sides (or a steep one) 0
        int tile_side = 0;
        float tile_slope = 0.f;
        if constexpr (BIAS) {
          tile_side = (q0 >= k0 + 127 || !n_ahead) ? 1 : (q0 + 127 <= k0 ? -1 : 0);
          if (fabsf(n_slope) > kSplitSlope) tile_side = 0;
          tile_slope = slope_log2(n_slope);
        }
        if (t < 64) {
          // -LSE in base 2, with the query's part of a one-sided bias
          float lv = -n_lse * kLog2e;
          if constexpr (BIAS) lv -= tile_side * tile_slope * static_cast<float>(q0 + 64 * w + t - k0);
          sLSE[64 * w + t] = lv;
          sDv[64 * w + t] = -n_dv / kDsUp;
          const int lo = min(max(n_see.x - k0, 0), 128), hi = min(max(n_see.y - k0, 0), 128);
          sSee[64 * w + t] = lo | (max(hi - lo, 0) << 16);
        }
        named_bar_sync(1 + w, 128);
        if (++i == I.ni) {
          i = 0;
          ++h;
        }
        if (it + 1 < I.niter) fetch(h, 128 * (I.i_begin + i));  // lands during this tile
        ok = mbar_wait(bar(C::BAR_S), par, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float4* sLSE4 = reinterpret_cast<const float4*>(sLSE);
        const uint4* sSee4 = reinterpret_cast<const uint4*>(sSee);
        // the key's part of a one-sided bias
        const float kb = BIAS ? tile_side * tile_slope * static_cast<float>(t) : 0.f;
        const uint64_t kb2 = f2_pack(kb, kb);
        uint32_t pk[2][16];  // fp16 pairs of P (1 - t^2) 2^15
#pragma unroll
        for (int hc = 0; hc < 2; ++hc) {
          const int cc = 2 * w + hc;  // 32-column chunk of the 128-column tile
          uint32_t s[32];
          tmem_ld32(lane_base + C::TM_S + 32 * cc, s);
          tmem_wait_ld(s);
          if constexpr (CAP) cap_scores(s, p.x_mul);  // s becomes t = tanh(x / cap)
          // Everything that depends on the tile is decided outside the column
          // loop (a branch in it, even one rarely taken, keeps the columns from
          // being scheduled together: 1477 us against 1172 at 2 x 16 x 8192 x 64).
          uint32_t pw[16];
          auto columns = [&](auto both_sides) {
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              const float4 l4 = sLSE4[8 * cc + m];
              const uint64_t s01 = f2_pack(__uint_as_float(s[4 * m + 0]), __uint_as_float(s[4 * m + 1]));
              const uint64_t s23 = f2_pack(__uint_as_float(s[4 * m + 2]), __uint_as_float(s[4 * m + 3]));
              uint64_t l01 = f2_pack(l4.x, l4.y), l23 = f2_pack(l4.z, l4.w);
              if constexpr (decltype(both_sides)::value) {  // |i - j| element by element
                const float d0 = static_cast<float>(q0 + 32 * cc + 4 * m - key);
                l01 = fsub2(l01, f2_pack(tile_slope * fabsf(d0), tile_slope * fabsf(d0 + 1.f)));
                l23 = fsub2(l23, f2_pack(tile_slope * fabsf(d0 + 2.f), tile_slope * fabsf(d0 + 3.f)));
              } else if constexpr (BIAS) {
                l01 = fadd2(l01, kb2);
                l23 = fadd2(l23, kb2);
              }
              const uint64_t y2 = CAP ? f2_pack(p.cap_log2, p.cap_log2) : c2;
              float x0, x1, x2, x3;
              f2_unpack(ffma2(s01, y2, l01), x0, x1);
              f2_unpack(ffma2(s23, y2, l23), x2, x3);
              const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
              pw[2 * m] = pack_bf16x2(p0, p1);
              pw[2 * m + 1] = pack_bf16x2(p2, p3);
              // P (1 - t^2) 2^15
              const uint64_t up = f2_pack(kDsUp, kDsUp), down = f2_pack(-kDsUp, -kDsUp);
              float a, b;
              f2_unpack(fmul2(f2_pack(p0, p1), CAP ? ffma2(fmul2(s01, down), s01, up) : up), a, b);
              pk[hc][2 * m] = pack_f16x2(a, b);
              f2_unpack(fmul2(f2_pack(p2, p3), CAP ? ffma2(fmul2(s23, down), s23, up) : up), a, b);
              pk[hc][2 * m + 1] = pack_f16x2(a, b);
            }
          };
          if constexpr (BIAS) {
            if (tile_side == 0) columns(std::true_type{});
            else columns(std::false_type{});
          } else {
            columns(std::false_type{});
          }
          if (!tile_full) {  // pairs outside the mask: 0 whatever they hold (a row without keys has LSE = -inf)
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              const uint4 sw = sSee4[8 * cc + m];
              auto seen = [&](uint32_t x) { return static_cast<uint32_t>(t) - (x & 0xffffu) < (x >> 16); };
              const uint32_t k01 = (seen(sw.x) ? 0xffffu : 0u) | (seen(sw.y) ? 0xffff0000u : 0u);
              const uint32_t k23 = (seen(sw.z) ? 0xffffu : 0u) | (seen(sw.w) ? 0xffff0000u : 0u);
              pw[2 * m] &= k01;
              pw[2 * m + 1] &= k23;
              pk[hc][2 * m] &= k01;
              pk[hc][2 * m + 1] &= k23;
            }
          }
          // P^T (bf16) into the first half of this warpgroup's own S^T columns
          tmem_st16(lane_base + C::TM_S + 64 * w + 16 * hc, pw);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::BAR_P));
        // dS^T = P^T (dP^T - D)
        ok = mbar_wait(bar(C::BAR_DP), par, abort_flag) && mbar_wait(bar(C::BAR_DS_EMPTY), par ^ 1u, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t region = sbase + C::OFF_DS + w * 16384;  // queries 64w..64w+63
        const float4* sDv4 = reinterpret_cast<const float4*>(sDv);
#pragma unroll
        for (int hc = 0; hc < 2; ++hc) {
          const int cc = 2 * w + hc;
          uint32_t dp[32];
          tmem_ld32(lane_base + C::TM_DP + 32 * cc, dp);
          tmem_wait_ld(dp);
          uint32_t wv[16];
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float4 d4 = sDv4[8 * cc + m];
            const uint32_t a0 = pk[hc][2 * m], a1 = pk[hc][2 * m + 1];
            float d0, d1, d2, d3;
            // (dP - D) 2^-15 times the kept factor: exact scalings
            const uint64_t dn = f2_pack(1.f / kDsUp, 1.f / kDsUp);
            const float2 g01 = __half22float2(*reinterpret_cast<const __half2*>(&a0));
            const float2 g23 = __half22float2(*reinterpret_cast<const __half2*>(&a1));
            f2_unpack(fmul2(f2_pack(g01.x, g01.y),
                            ffma2(f2_pack(__uint_as_float(dp[4 * m + 0]), __uint_as_float(dp[4 * m + 1])), dn,
                                  f2_pack(d4.x, d4.y))), d0, d1);
            f2_unpack(fmul2(f2_pack(g23.x, g23.y),
                            ffma2(f2_pack(__uint_as_float(dp[4 * m + 2]), __uint_as_float(dp[4 * m + 3])), dn,
                                  f2_pack(d4.z, d4.w))), d2, d3);
            wv[2 * m] = pack_bf16x2(d0, d1);
            wv[2 * m + 1] = pack_bf16x2(d2, d3);
          }
          // 32 queries -> 16-byte chunks hc*4 + 0..3 of this row in region w
#pragma unroll
          for (int u = 0; u < 4; ++u)
            st_shared_v4(region + sw128_offset(t, hc * 4 + u), wv[4 * u], wv[4 * u + 1], wv[4 * u + 2], wv[4 * u + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(C::BAR_DS));
      }
      if (!ok) break;
      // this item's rows: warpgroup 0 stores dK (times scale), warpgroup 1 stores
      // dV, then both hand the accumulator columns back to the next item
      const bool any = I.niter > 0;  // else: a key tile no query sees, stored as zero
      if (any) {
        ok = mbar_wait(bar(C::BAR_ACC), nitems & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
      }
      const size_t row = (static_cast<size_t>(I.b) * p.N + key) * p.Hkv + I.hk;
      const uint32_t col = w ? C::TM_DV : C::TM_DK;
      const float mul = w ? 1.f : p.scale;
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(w ? p.dv : p.dk) + row * D;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t a[32];
        if (any) {
          tmem_ld32(lane_base + col + 32 * cc, a);
          tmem_wait_ld(a);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = 0u;
        }
        if (p.dk_part) {  // uniform over the grid
          if (key_ok) {
            float* part = (w ? p.dv_part : p.dk_part) +
                          ((static_cast<size_t>(I.b) * p.N + key) * p.Hv + I.hv) * D + 32 * cc;
#pragma unroll
            for (int u = 0; u < 8; ++u) st_global_v4(part + 4 * u, a[4 * u], a[4 * u + 1], a[4 * u + 2], a[4 * u + 3]);
          }
          continue;
        }
        uint32_t wv[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          wv[i] = pack_bf16x2(__uint_as_float(a[2 * i]) * mul, __uint_as_float(a[2 * i + 1]) * mul);
        if (key_ok) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            st_global_v4(dst + 32 * cc + 8 * u, wv[4 * u], wv[4 * u + 1], wv[4 * u + 2], wv[4 * u + 3]);
        }
      }
      if (any) {
        tc_fence_before();
        mbar_arrive(bar(C::BAR_ACC_FREE));
        gt0 += I.niter;
        ++nitems;
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ dQ_i drain
    regs_set<C::REGS_DRAIN, C::LAUNCH_REGS>();
    const int t = threadIdx.x - 256;  // query row within the tile == tensor-memory lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int gt0 = 0;
    for (int n = 0;; ++n) {
      bool ok;
      const int item = take_item(n, ok);
      if (!__all_sync(0xffffffffu, ok) || item < 0) break;
      ModBwdItem I;
      mod_bwd_item(p, item, I);
      if constexpr (DQ) {
        int h = I.hv * p.hs, i = 0;
        for (int it = 0; it < I.niter; ++it) {
          const uint32_t par = (gt0 + it) & 1;
          const int q = 128 * (I.i_begin + i) + t;
          ok = mbar_wait(bar(C::BAR_DQ_FULL), par, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // accumulator rows: (bh, float4 group g, r) with r consecutive across the warp
          const int bh_ = I.b * p.H + h;
          if (++i == I.ni) {
            i = 0;
            ++h;
          }
          float4* acc4 = reinterpret_cast<float4*>(p.dq_acc);
          // The whole dQ_i row is loaded first and its tensor-memory columns are
          // released at once (at d = 128 dP^T(i+1) reuses them); the atomics
          // then run from registers.  Issuing atomics stalls once the memory
          // pipeline backs up, so none may stand between dQ_i and dP^T(i+1).
          uint32_t a[D / 32][32];
#pragma unroll
          for (int cg = 0; cg < D / 32; ++cg) tmem_ld32(lane_base + C::TM_DQ + 32 * cg, a[cg]);
#pragma unroll
          for (int cg = 0; cg < D / 32; ++cg) tmem_wait_ld(a[cg]);
          tc_fence_before();
          mbar_arrive(bar(C::BAR_DQ_EMPTY));
          if (q < p.N) {
#pragma unroll
            for (int cg = 0; cg < D / 32; ++cg)
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                atomicAdd(acc4 + dq_acc_index4(bh_, 8 * cg + u, q, p.N, D),
                          make_float4(__uint_as_float(a[cg][4 * u]), __uint_as_float(a[cg][4 * u + 1]),
                                      __uint_as_float(a[cg][4 * u + 2]), __uint_as_float(a[cg][4 * u + 3])));
                if (u & 1) {
                  const long long t0 = clock64();
                  while (clock64() - t0 < C::DQ_ATOMIC_PAUSE) {
                  }
                }
              }
          }
        }
        if (!ok) break;
      }
      gt0 += I.niter;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// What is left after the main kernel, in one launch.  Blocks below nconv: dQ to
// bf16.  The others, where a group's heads were split: dK = scale * sum, dV = sum
// of the group's partial sums, in the order of the heads; one thread per four
// columns, first the keys, then the values.
template <int D>
__global__ void __launch_bounds__(256) fa_mod_bwd_finish_kernel(const ModBwdParams p, unsigned nconv, unsigned nred) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the main kernel has ended and its sums are visible
  if (blockIdx.x < nconv) {  // 32 rows of one head, through shared memory as in fa_bwd_dq_convert_kernel
    constexpr int G4 = D / 4, CPR = D / 8;
    __shared__ float4 tile[32][G4 + 1];
    const unsigned nblk = (static_cast<unsigned>(p.N) + 31u) / 32u;
    const int bh = static_cast<int>(blockIdx.x / nblk), r0 = static_cast<int>(blockIdx.x % nblk) * 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const float4* acc = reinterpret_cast<const float4*>(p.dq_acc);
#pragma unroll
    for (int g = w; g < G4; g += 8)
      if (r0 + lane < p.N) tile[lane][g] = __ldcs(acc + dq_acc_index4(bh, g, r0 + lane, p.N, D));
    __syncthreads();
    const int h = bh % p.H, b = bh / p.H;
    uint4* dst = reinterpret_cast<uint4*>(p.dq) + ((static_cast<size_t>(b) * p.N + r0) * p.H + h) * CPR;
#pragma unroll
    for (int e = threadIdx.x; e < 32 * CPR; e += 256) {
      const int r = e / CPR, c = e % CPR;
      if (r0 + r >= p.N) continue;
      const float4 x = tile[r][2 * c], y = tile[r][2 * c + 1];
      __stcs(dst + static_cast<size_t>(r) * p.H * CPR + c,
             make_uint4(pack_bf16x2(x.x * p.scale, x.y * p.scale), pack_bf16x2(x.z * p.scale, x.w * p.scale),
                        pack_bf16x2(y.x * p.scale, y.y * p.scale), pack_bf16x2(y.z * p.scale, y.w * p.scale)));
    }
    return;
  }
  const int64_t n4 = static_cast<int64_t>(p.B) * p.N * p.Hkv * (D / 4);
  unsigned blk = blockIdx.x - nconv;
  const bool values = blk >= nred;
  if (values) blk -= nred;
  const int64_t i = static_cast<int64_t>(blk) * 256 + threadIdx.x;
  if (i >= n4) return;
  const int parts = p.Hv / p.Hkv, q = D / 4;
  const int64_t row = i / q;  // (token, key head); its partials are rows row * parts ..
  const float4* src = reinterpret_cast<const float4*>(values ? p.dv_part : p.dk_part) + row * parts * q + i % q;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const float4 v = __ldcs(src + static_cast<int64_t>(k) * q);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  const float mul = values ? 1.f : p.scale;
  reinterpret_cast<uint2*>(values ? p.dv : p.dk)[i] =
      make_uint2(pack_bf16x2(a.x * mul, a.y * mul), pack_bf16x2(a.z * mul, a.w * mul));
}

}  // namespace fa
