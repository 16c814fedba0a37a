// Decoding from the 8-bit cache (fa_cache.cuh) for sm_100a: a few new queries
// per sequence, grouped heads, with the score cap, distance bias and window of
// the modified-score attention.
//
//     x_ij = scale q_i . k_j,  k_j = 2^(ek_j - 127) codes
//     z_ij = cap tanh(x_ij / cap) - slope_h |pos_i - j|,  pos_i = L - Nq + i
//     O_i  = sum_j softmax_j(z_ij) v_j
// over the keys j < L, with causal j <= pos_i, with a window |pos_i - j| < W.
//
// The cache is read once, so the bound is HBM: 2 (d + 1) bytes per key and key
// head.  At 6.5 TB/s an SM receives a 256-byte key/value pair every ~11 clocks,
// too little time to convert and multiply 256 codes per query row on the CUDA
// cores, so both products are tensor-core ones (mma m16n8k16, fp16 operands,
// fp32 sums): the G Nq query rows of a key head fill up to 16 rows.  tcgen05
// is not used: its operands come from shared memory, where codes would have to
// be written back as 16-bit values first, and its smallest M is four times the
// rows there are.
//   - e4m3 is exact in fp16.  A query row is scaled by a power of two to just
//     under 2^15 and is then exact in fp16 down to 2^-24 (its 8 significant
//     bits fit); row scale and key scale are applied to the fp32 score.
//   - The weight of key j in the second product is w_ij = 2^(z_ij + ev_j - mo_i)
//     in fp16 (error 2^-11 relative, an eighth of the output's rounding to bf16):
//     the value row's exponent ev_j joins the weight's, with a running maximum
//     mo_i of its own, so w <= 2^8 and the largest contribution keeps full
//     precision whatever the spread of the value scales.  The row sum is taken
//     of 2^(z_ij - m_i) unrounded in fp32.
//   - Operand layout: a k-step may take the head dimensions, and the second
//     product's output columns, in any order as long as both operands agree.
//     Thread (g, t) of a warp takes 32 contiguous dimensions of key g for the
//     scores and 16 contiguous dimensions of keys 2t, 2t+1, 2t+8, 2t+9 for the
//     output: 16-byte shared-memory loads, conflict-free under TMA's 128-byte
//     swizzle at d = 128; no transposition of V.
//   - Each of the four compute warps owns 16 keys of a 64-key tile with its own
//     running maxima, sums and output: no block-wide step per tile.  They are
//     joined in shared memory at the end of a segment piece.
// Work split: as fa_decode.cuh, stream-K over (batch entry, key head, row
// block, 64-key tile) units in equal contiguous chunks, partial records of
// shared segments merged through their logsumexps by a second kernel.  Each CTA
// finds its chunk by scanning the lengths itself: no prefix launch.
#pragma once
#include "fa_cache.cuh"
#include "fa_mod_fwd.cuh"

namespace fa {

constexpr int kCacheDecodeGrid = 2 * 148;

struct CDecParams {
  const void* q;          // bf16 [B, Nq, H, d]
  void* o;                // bf16 [B, Nq, H, d]
  float* lse;             // [B, H, Nq]
  const uint8_t* kexp;    // [B, Hkv, Nk]
  const uint8_t* vexp;
  const int* seqlens;     // [B] or nullptr
  const float* slopes;    // [H] or nullptr
  long long* prefix;      // [B + 1] first unit of each entry, for the merge
  int* bad;
  float* rec_o;           // [grid][2][16][d]
  float* rec_lse;         // [grid][2][16]
  int B, Nq, Nk, H, Hkv, G;
  int rows, nrb;          // G Nq query rows per key head, blocks of 16
  int grid, causal, window;
  float scale_log2;       // scale log2 e          (no cap)
  float x_mul, cap_log2;  // scale / cap, cap log2 e
};

template <int D>
struct CDecCfg {
  static constexpr int KT = 64;
  static constexpr int NW = 4;                     // compute warps, 16 keys of a tile each
  static constexpr int TILE = KT * D;              // bytes of a K or V tile
  static constexpr int NSTAGE = D == 128 ? 6 : 10;
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_SC = OFF_KV + NSTAGE * 2 * TILE;   // float [NW][2][32] key and value scales
  static constexpr int OFF_ML = OFF_SC + NW * 2 * 32 * 4;     // float [3][NW][16] m, mo, l
  static constexpr int OFF_ACC = OFF_ML + 3 * NW * 16 * 4;    // float [NW][4][D + 4]
  static constexpr int ACC_LD = D + 4;
  static constexpr int OFF_BAR = OFF_ACC + NW * 4 * ACC_LD * 4;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = NSTAGE, NBAR = 2 * NSTAGE;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  // misc: abort flag | bad | scan [8] | b0 | base of b0 (8 bytes) | U (8 bytes)
  static constexpr int SMEM_BYTES = OFF_MISC + 128 + 1024;
  static constexpr int THREADS = 32 * (NW + 1);
  static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "two CTAs per SM");
};

// First and one-past-last 64-key tile that any query of an entry of length L
// sees, and the units they make.
struct CDecRange {
  int t0, t1;
};
__device__ __forceinline__ CDecRange cdec_range(const CDecParams& p, int L) {
  CDecRange r;
  r.t1 = (L + 63) >> 6;
  const int first = p.window > 0 && p.window < p.Nk ? max(0, L - p.Nq - p.window + 1) : 0;
  r.t0 = min(first >> 6, r.t1);
  return r;
}
__device__ __forceinline__ int cdec_len(const CDecParams& p, int b) { return p.seqlens ? p.seqlens[b] : p.Nk; }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(160, 2)
    fa_cache_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const CDecParams p) {
  using C = CDecCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int n) -> uint32_t { return sbase + C::OFF_BAR + 8u * n; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  int* s_bad = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);
  long long* s_scan = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);  // [5]
  int* s_b0 = reinterpret_cast<int*>(smem + C::OFF_MISC + 56);
  long long* s_base0 = reinterpret_cast<long long*>(smem + C::OFF_MISC + 64);
  int* s_ok = reinterpret_cast<int*>(smem + C::OFF_MISC + 72);  // [4] per compute warp

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NSTAGE; ++s) {
      mbar_init(bar(C::BAR_FULL + s), 1);
      mbar_init(bar(C::BAR_EMPTY + s), C::NW * 32);
    }
    *abort_flag = 0;
    *s_bad = 0;
    fence_mbar_init();
  }
  __syncthreads();

  // ---- this CTA's units: every thread sums a run of entries, block scan
  const int per = (p.B + C::THREADS - 1) / C::THREADS;
  const int e0 = min(p.B, static_cast<int>(threadIdx.x) * per), e1 = min(p.B, e0 + per);
  auto units = [&](int b) -> long long {
    const int L = cdec_len(p, b);
    if (L < 0 || L > p.Nk) return -1;
    const CDecRange r = cdec_range(p, L);
    return static_cast<long long>(r.t1 - r.t0) * p.Hkv * p.nrb;
  };
  long long sum = 0;
  bool bad = false;
  for (int b = e0; b < e1; ++b) {
    const long long x = units(b);
    if (x < 0) bad = true;
    else sum += x;
  }
  if (bad) *s_bad = 1;
  long long inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += x;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  long long U = 0, base = inc - sum;
  for (int w = 0; w < C::NW + 1; ++w) {
    if (w < warp) base += s_scan[w];
    U += s_scan[w];
  }
  const bool any_bad = *s_bad != 0;
  const long long chunk = (U + p.grid - 1) / p.grid;
  const long long u0 = static_cast<long long>(blockIdx.x) * chunk;
  const long long u1 = min(U, u0 + chunk);
  if (blockIdx.x == 0) {  // the merge kernel's copy
    long long run = base;
    for (int b = e0; b < e1; ++b) {
      p.prefix[b] = run;
      const long long x = units(b);
      run += x < 0 ? 0 : x;
    }
    if (threadIdx.x == 0) {
      p.prefix[p.B] = U;
      *p.bad = any_bad;
      if (any_bad) atomicOr(&g_fa_error_word, FA_DEVERR_BOUNDS);
    }
  }
  if (any_bad) return;  // lengths contradict the cache: write nothing
  if (u0 >= u1) return;  // uniform over the CTA
  if (base <= u0 && u0 < base + sum) {
    long long run = base;
    int b = e0;
    for (;;) {
      const long long x = units(b);
      if (u0 < run + x) break;
      run += x;
      ++b;
    }
    *s_b0 = b;
    *s_base0 = run;
  }
  __syncthreads();

  // Walk of the units [u0, u1), the same in both roles: segment (b, hk, rb),
  // its tiles [r.t0, r.t1), the current tile tp.
  struct Walk {
    int b, hk, rb, tp, L;
    CDecRange r;
  };
  auto walk_begin = [&](Walk& w) {
    w.b = *s_b0;
    w.L = cdec_len(p, w.b);
    w.r = cdec_range(p, w.L);
    const long long rel = u0 - *s_base0;
    const int T = w.r.t1 - w.r.t0;
    const int seg = static_cast<int>(rel / T);
    w.tp = w.r.t0 + static_cast<int>(rel % T);
    w.hk = seg / p.nrb;
    w.rb = seg % p.nrb;
  };
  auto walk_next = [&](Walk& w) {  // after the last tile of a segment, with units left
    if (++w.rb == p.nrb) {
      w.rb = 0;
      if (++w.hk == p.Hkv) {
        w.hk = 0;
        do {
          ++w.b;
          w.L = cdec_len(p, w.b);
          w.r = cdec_range(p, w.L);
        } while (w.r.t0 >= w.r.t1);
      }
    }
    w.tp = w.r.t0;
  };

  if (warp == C::NW) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      Walk w;
      walk_begin(w);
      int issued = 0;
      bool ok = true;
      for (long long u = u0; ok && u < u1; ++u) {
        const int st = issued % C::NSTAGE;
        if (!(ok = mbar_wait(bar(C::BAR_EMPTY + st), ((issued / C::NSTAGE) & 1) ^ 1u, abort_flag))) break;
        const int row = w.tp * C::KT;
        const int boxes = w.L - row > 32 ? 2 : 1;  // boxes of 32 keys; none past the length
        mbar_arrive_expect_tx(bar(C::BAR_FULL + st), boxes * 2 * 32 * D);
        const uint32_t dst = sbase + C::OFF_KV + st * 2 * C::TILE;
        for (int x = 0; x < boxes; ++x) {
          tma_load_4d(dst + x * 32 * D, &tmK, bar(C::BAR_FULL + st), 0, w.hk, row + 32 * x, w.b);
          tma_load_4d(dst + C::TILE + x * 32 * D, &tmV, bar(C::BAR_FULL + st), 0, w.hk, row + 32 * x, w.b);
        }
        ++issued;
        if (++w.tp == w.r.t1 && u + 1 < u1) walk_next(w);
      }
      if (*abort_flag) {  // let the copies in flight land before the CTA exits
        for (int n = 0; n < C::NSTAGE && n < issued; ++n) {
          const int m = issued - 1 - n;
          mbar_wait_drain(bar(C::BAR_FULL + m % C::NSTAGE), (m / C::NSTAGE) & 1);
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- compute
  const int g = lane >> 2, t = lane & 3;
  constexpr int KS = D / 16;      // k-steps of the scores
  constexpr int ND = D / 8;       // output columns per (g): n-tiles of the second product
  float* sSc = reinterpret_cast<float*>(smem + C::OFF_SC) + warp * 64;
  float* sMl = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* sAcc = reinterpret_cast<float*>(smem + C::OFF_ACC);
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kLazy = 8.f;    // the maxima move when exceeded by more than 2^8
  int gtile = 0;
  Walk w;
  walk_begin(w);
  for (long long u = u0; u < u1;) {
    const int n = static_cast<int>(min(static_cast<long long>(w.r.t1 - w.tp), u1 - u));
    const int L = w.L;
    // ---- query rows g and g + 8 of this row block: thread t takes D / 4
    // contiguous dimensions; scaled by 2^-a to below 2^15
    uint32_t qa[KS][4];
    float rowf[2];                 // score factor of the row
    float slope[2] = {0.f, 0.f};
    int pos[2];                    // the query's position
    bool row_ok[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = w.rb * 16 + g + 8 * e;
      row_ok[e] = r < p.rows;
      const int qi = row_ok[e] ? r / p.G : 0, h = w.hk * p.G + (row_ok[e] ? r % p.G : 0);
      pos[e] = L - p.Nq + qi;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(p.q) + ((static_cast<size_t>(w.b) * p.Nq + qi) * p.H + h) * D + t * (D / 4));
      uint32_t x[D / 8];
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = row_ok[e] ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        x[4 * i] = v.x;
        x[4 * i + 1] = v.y;
        x[4 * i + 2] = v.z;
        x[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) a = fmaxf(a, fmaxf(fabsf(bf16lo_to_f32(x[i])), fabsf(bf16hi_to_f32(x[i]))));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
      // 2^ea: exponent that brings a below 2^15 (0 stays 0; subnormals gain at most 2^120)
      const int ea = a > 0.f ? max(static_cast<int>(__float_as_uint(a) >> 23) - 127 - 14, -120) : 0;
      const float mul = __uint_as_float(static_cast<uint32_t>(127 - ea) << 23);
      rowf[e] = (CAP ? p.x_mul : p.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + ea) << 23);
      if (BIAS) slope[e] = p.slopes[h] * kLog2e;
#pragma unroll
      for (int s = 0; s < KS; ++s) {  // k-step s: this thread's dimensions 4s .. 4s + 3
        qa[s][e] = pack_h2(bf16lo_to_f32(x[2 * s]) * mul, bf16hi_to_f32(x[2 * s]) * mul);
        qa[s][2 + e] = pack_h2(bf16lo_to_f32(x[2 * s + 1]) * mul, bf16hi_to_f32(x[2 * s + 1]) * mul);
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, mo[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float acc[ND][4];
#pragma unroll
    for (int c = 0; c < ND; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;

    // scale bytes of this warp's 16 keys, one lane each (lanes 16-31: values),
    // fetched one tile ahead
    const uint8_t* exps = (lane < 16 ? p.kexp : p.vexp) + (static_cast<size_t>(w.b) * p.Hkv + w.hk) * p.Nk;
    auto fetch_exp = [&](int tile) -> uint32_t {
      const int key = tile * C::KT + warp * 16 + (lane & 15);
      return key < L ? exps[key] : 127u;
    };
    uint32_t ex = fetch_exp(w.tp);
    // keys that some query of the entry sees
    const int key_lo = p.window > 0 && p.window < p.Nk ? L - p.Nq - p.window + 1 : 0;
    bool ok = true;
    for (int it = 0; it < n; ++it, ++gtile) {
      const int st = gtile % C::NSTAGE;
      const int k0 = (w.tp + it) * C::KT + warp * 16;  // this warp's first key
      __syncwarp();
      // keys: the scale itself; values: its exponent
      sSc[lane] = lane < 16 ? e8m0_value(ex) : (ex == 255u ? __uint_as_float(0x7fffffffu) : static_cast<float>(ex) - 127.f);
      if (it + 1 < n) ex = fetch_exp(w.tp + it + 1);
      __syncwarp();
      ok = mbar_wait(bar(C::BAR_FULL + st), (gtile / C::NSTAGE) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint8_t* pK = smem + C::OFF_KV + st * 2 * C::TILE + warp * 16 * D;
      const uint8_t* pV = pK + C::TILE;
      if (k0 < L) {  // warp-uniform
        // ---- scores: two n-tiles of 8 keys
        float sc[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          sc[x][0] = sc[x][1] = sc[x][2] = sc[x][3] = 0.f;
          const int r = 8 * x + g;  // key row within the warp's 16
          uint32_t kw[KS];
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            // 16-byte chunk (D / 64) t + i of the row, swizzled as TMA wrote it
            const int ch = (D == 128) ? ((2 * t + i) ^ (r & 7)) : (t ^ ((r >> 1) & 3));
            const uint4 v = *reinterpret_cast<const uint4*>(pK + r * D + ch * 16);
            kw[4 * i] = v.x;
            kw[4 * i + 1] = v.y;
            kw[4 * i + 2] = v.z;
            kw[4 * i + 3] = v.w;
          }
#pragma unroll
          for (int s = 0; s < KS; ++s)
            mma_f16(sc[x], qa[s][0], qa[s][1], qa[s][2], qa[s][3], e4m3x2_to_h2(kw[s]), e4m3x2_to_h2(kw[s] >> 16));
        }
        // ---- z in base 2, mask, maxima.  Element c: row g + 8 (c >> 1), key
        // 8x + 2t + (c & 1)
        float mx[2] = {-INFINITY, -INFINITY}, mxo[2] = {-INFINITY, -INFINITY};
        float so[2][4];  // z + ev: exponent of the weight; a select, so that an
                         // unseen key's scale (NaN perhaps) stays out
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 ks = *reinterpret_cast<const float2*>(sSc + 8 * x + 2 * t);
          const float2 vs = *reinterpret_cast<const float2*>(sSc + 16 + 8 * x + 2 * t);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int e = c >> 1;
            const int key = k0 + 8 * x + 2 * t + (c & 1);
            float z = sc[x][c] * rowf[e] * ((c & 1) ? ks.y : ks.x);
            if (CAP) z = p.cap_log2 * tanh_any(z);
            const int away = pos[e] - key;
            if (BIAS) z = fmaf(-slope[e], fabsf(static_cast<float>(away)), z);
            const bool see = key < L && (!p.causal || away >= 0) &&
                             (p.window <= 0 || (away < p.window && -away < p.window));
            sc[x][c] = see ? z : -INFINITY;
            so[x][c] = see ? z + ((c & 1) ? vs.y : vs.x) : -INFINITY;
            mx[e] = fmaxf(mx[e], sc[x][c]);
            mxo[e] = fmaxf(mxo[e], so[x][c]);
          }
        }
        bool move = false;
        float al[2], alo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mxo[e] = fmaxf(mxo[e], __shfl_xor_sync(0xffffffffu, mxo[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          mxo[e] = fmaxf(mxo[e], __shfl_xor_sync(0xffffffffu, mxo[e], 2));
          al[e] = alo[e] = 1.f;
          if (mx[e] > m[e] + kLazy || (m[e] == -INFINITY && mx[e] > -INFINITY)) {
            al[e] = ex2(m[e] - mx[e]);
            m[e] = mx[e];
          }
          if (mxo[e] > mo[e] + kLazy || (mo[e] == -INFINITY && mxo[e] > -INFINITY)) {
            alo[e] = ex2(mo[e] - mxo[e]);
            mo[e] = mxo[e];
            move = true;
          }
          l[e] *= al[e];
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int c = 0; c < ND; ++c) {
            acc[c][0] *= alo[0];
            acc[c][1] *= alo[0];
            acc[c][2] *= alo[1];
            acc[c][3] *= alo[1];
          }
        }
        // ---- weights: A operand of the second product
        uint32_t wa[4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float nm = m[e] == -INFINITY ? 0.f : -m[e], nmo = mo[e] == -INFINITY ? 0.f : -mo[e];
            l[e] += ex2(sc[x][2 * e] + nm) + ex2(sc[x][2 * e + 1] + nm);
            wa[2 * x + e] = pack_h2(ex2(so[x][2 * e] + nmo), ex2(so[x][2 * e + 1] + nmo));
          }
        // ---- output: keys 2t, 2t+1 (first half of k) and 2t+8, 2t+9
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * t + (i & 1) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(pV + r * D + ((g ^ (r & 7)) << 4));
            vw[i][0] = v.x;
            vw[i][1] = v.y;
            vw[i][2] = v.z;
            vw[i][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(pV + r * D + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
            vw[i][0] = v.x;
            vw[i][1] = v.y;
          }
        }
        if (k0 + 16 > L || k0 < key_lo) {  // rows no query sees may hold NaN codes: 0 x NaN
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = k0 + 2 * t + (i & 1) + 8 * (i >> 1);
            if (key >= L || key < key_lo)
#pragma unroll
              for (int c = 0; c < D / 32; ++c) vw[i][c] = 0u;
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // four output columns at a time
          // bytes (key, key + 1) of columns 4c .. 4c + 3
          const uint32_t a01 = __byte_perm(vw[0][c], vw[1][c], 0x5140), a23 = __byte_perm(vw[0][c], vw[1][c], 0x7362);
          const uint32_t b01 = __byte_perm(vw[2][c], vw[3][c], 0x5140), b23 = __byte_perm(vw[2][c], vw[3][c], 0x7362);
          mma_f16(acc[4 * c + 0], wa[0], wa[1], wa[2], wa[3], e4m3x2_to_h2(a01), e4m3x2_to_h2(b01));
          mma_f16(acc[4 * c + 1], wa[0], wa[1], wa[2], wa[3], e4m3x2_to_h2(a01 >> 16), e4m3x2_to_h2(b01 >> 16));
          mma_f16(acc[4 * c + 2], wa[0], wa[1], wa[2], wa[3], e4m3x2_to_h2(a23), e4m3x2_to_h2(b23));
          mma_f16(acc[4 * c + 3], wa[0], wa[1], wa[2], wa[3], e4m3x2_to_h2(a23 >> 16), e4m3x2_to_h2(b23 >> 16));
        }
      }
      mbar_arrive(bar(C::BAR_EMPTY + st));
    }
    // ---- join the four warps: rows of the block in passes of four
    if (lane == 0) s_ok[warp] = ok;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (t == 0) {
        sMl[(0 * C::NW + warp) * 16 + g + 8 * e] = m[e];
        sMl[(1 * C::NW + warp) * 16 + g + 8 * e] = mo[e];
        sMl[(2 * C::NW + warp) * 16 + g + 8 * e] = l[e];
      }
    }
    named_bar_sync(1, C::NW * 32);
    // a wait gave up in some warp: the error word is set; write nothing more
    // (every warp reads the same four flags, so all of them leave)
    if (!(s_ok[0] && s_ok[1] && s_ok[2] && s_ok[3])) return;
    const bool whole = w.tp == w.r.t0 && n == w.r.t1 - w.r.t0;  // the piece is the whole segment
    const int slot = (u == u0) ? 0 : 1;
    const int nrows = min(16, p.rows - w.rb * 16);
    float f[2];  // this warp's output factor per row: 2^(mo_w - mo), 0 when it saw nothing
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float M = -INFINITY;
      for (int x = 0; x < C::NW; ++x) M = fmaxf(M, sMl[(C::NW + x) * 16 + g + 8 * e]);
      f[e] = mo[e] == -INFINITY ? 0.f : ex2(mo[e] - M);
    }
    for (int r0 = 0; r0 < nrows; r0 += 4) {
      // rows r0 .. r0 + 3: lanes g = r0 % 8 .. + 3, half e = r0 / 8
      const int e = r0 >> 3;
      if ((g & 4) == (r0 & 4)) {
        float* dst = sAcc + (warp * 4 + (g & 3)) * C::ACC_LD + t * (D / 4);
        const float fe = e ? f[1] : f[0];
#pragma unroll
        for (int c = 0; c < ND; ++c) {
          // column 2t, 2t + 1 of n-tile c: dimensions (2t) ND + c and (2t + 1) ND + c
          dst[c] = (e ? acc[c][2] : acc[c][0]) * fe;
          dst[ND + c] = (e ? acc[c][3] : acc[c][1]) * fe;
        }
      }
      named_bar_sync(1, C::NW * 32);
      const int rr = threadIdx.x >> 5;  // warp = row of the pass
      const int row = r0 + rr;
      if (row < nrows) {
        float M = -INFINITY, MO = -INFINITY, lsum = 0.f;
#pragma unroll
        for (int x = 0; x < C::NW; ++x) {
          M = fmaxf(M, sMl[x * 16 + row]);
          MO = fmaxf(MO, sMl[(C::NW + x) * 16 + row]);
        }
#pragma unroll
        for (int x = 0; x < C::NW; ++x) {
          const float mw = sMl[x * 16 + row];
          if (mw != -INFINITY) lsum += sMl[(2 * C::NW + x) * 16 + row] * ex2(mw - M);
          else if (sMl[(2 * C::NW + x) * 16 + row] != 0.f) lsum = sMl[(2 * C::NW + x) * 16 + row];  // NaN scores
        }
        const float inv = lsum == 0.f ? 0.f : ex2(MO - M) / lsum;
        const float lse = lsum == 0.f ? -INFINITY : (M + lg2(lsum)) * kLn2;
        const int r = w.rb * 16 + row, qi = r / p.G, h = w.hk * p.G + r % p.G;
        const size_t rec = (static_cast<size_t>(blockIdx.x) * 2 + slot) * 16 + row;
        for (int c = lane * 2; c < D; c += 64) {
          float a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int x = 0; x < C::NW; ++x) {
            const float2 v = *reinterpret_cast<const float2*>(sAcc + (x * 4 + rr) * C::ACC_LD + c);
            a0 += v.x;
            a1 += v.y;
          }
          a0 *= inv;
          a1 *= inv;
          if (whole)
            *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) +
                                         ((static_cast<size_t>(w.b) * p.Nq + qi) * p.H + h) * D + c) = pack_bf16x2(a0, a1);
          else
            *reinterpret_cast<float2*>(p.rec_o + rec * D + c) = make_float2(a0, a1);
        }
        if (lane == 0) {
          if (whole) p.lse[(static_cast<size_t>(w.b) * p.H + h) * p.Nq + qi] = lse;
          else p.rec_lse[rec] = lse;
        }
      }
      named_bar_sync(1, C::NW * 32);
    }
    u += n;
    w.tp += n;
    if (w.tp == w.r.t1 && u < u1) walk_next(w);
  }
}

// One warp per output row (batch entry, head, query): rows of entries whose
// queries see no tile get O = 0, LSE = -inf; rows of segments shared by
// several CTAs are combined from their records; the rest is written already.
__global__ void __launch_bounds__(128) fa_cache_decode_merge_kernel(const CDecParams p, int D) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + warp;
  const long long nrows = static_cast<long long>(p.B) * p.H * p.Nq;
  if (row >= nrows || *p.bad) return;
  const int qi = static_cast<int>(row % p.Nq);
  const long long bh = row / p.Nq;
  const int b = static_cast<int>(bh / p.H), h = static_cast<int>(bh % p.H);
  const CDecRange rg = cdec_range(p, cdec_len(p, b));
  const int T = rg.t1 - rg.t0;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + ((static_cast<size_t>(b) * p.Nq + qi) * p.H + h) * D;
  float* lse = p.lse + bh * p.Nq + qi;
  if (T == 0) {
    for (int c = lane; c < D; c += 32) out[c] = __float2bfloat16(0.f);
    if (lane == 0) *lse = -INFINITY;
    return;
  }
  const long long U = p.prefix[p.B];
  const long long chunk = (U + p.grid - 1) / p.grid;
  const int r = qi * p.G + h % p.G;  // row of its key head
  const long long s0 = p.prefix[b] + (static_cast<long long>(h / p.G) * p.nrb + (r >> 4)) * T, s1 = s0 + T;
  const int g0 = static_cast<int>(s0 / chunk), g1 = static_cast<int>((s1 - 1) / chunk);
  if (g0 == g1) return;
  const int n = g1 - g0 + 1;
  // CTA g0's piece is its last one (slot 1) unless its chunk starts with the
  // segment; every later CTA's piece is its first one (slot 0)
  const int slot0 = static_cast<long long>(g0) * chunk < s0 ? 1 : 0;
  auto rec = [&](int k) -> size_t { return (static_cast<size_t>(g0 + k) * 2 + (k == 0 ? slot0 : 0)) * 16 + (r & 15); };
  float mx = -INFINITY;
  bool nan = false;
  for (int k = lane; k < n; k += 32) {
    const float x = p.rec_lse[rec(k)];
    nan |= x != x;
    mx = fmaxf(mx, x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  nan = __any_sync(0xffffffffu, nan);
  constexpr float kLog2ef = 1.4426950408889634f;
  float den = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < n; ++k) {
    const float lr = p.rec_lse[rec(k)];
    if (lr == -INFINITY) continue;
    const float wk = ex2((lr - mx) * kLog2ef);
    den += wk;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < D) acc[c] = fmaf(wk, p.rec_o[rec(k) * D + lane + 32 * c], acc[c]);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < D) out[lane + 32 * c] = __float2bfloat16(acc[c] * inv);
  if (lane == 0) *lse = nan ? __uint_as_float(0x7fffffffu) : (den == 0.f ? -INFINITY : mx + lg2(den) * kLn2);
}

}  // namespace fa
