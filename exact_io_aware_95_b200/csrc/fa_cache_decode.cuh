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
// fp32 sums), with the cache as the 16-row operand and the G Nq query rows of a
// key head as the 8 columns (NB = 1) or two times 8 (NB = 2; more rows take
// further passes over the cache).  tcgen05 is not used: its operands come from
// shared memory, where codes would have to be written back as 16-bit values
// first, and its smallest M is many times the rows there are.
//   - e4m3 is exact in fp16.  A query row is scaled by a power of two to just
//     under 2^15 and is then exact in fp16 down to 2^-24 (its 8 significant
//     bits fit); row scale and key scale are applied to the fp32 score.
//   - The weight of key j in the second product is w_ij = 2^(z_ij + ev_j - mo_i)
//     in fp16 (error 2^-11 relative, an eighth of the output's rounding to bf16; half
//     a step of 2^-24 where the weight is below 2^-14 of the one that set mo_i):
//     the value row's exponent ev_j joins the weight's, with a running maximum
//     mo_i of its own, so the largest contribution keeps full precision whatever
//     the spread of the value scales.  The row sum is taken of 2^(z_ij - m_i)
//     unrounded in fp32.  Both maxima move only when a score exceeds them by
//     more than 8 (w <= 2^8 fits fp16): a warp votes on that, and reduces a new
//     maximum over its lanes only then, so most tiles need no shuffles.
//   - Operand layout: a k-step may take the head dimensions, and the second
//     product's rows, in any order as long as both operands agree.  Thread
//     (g, t) of a warp takes D / 4 contiguous dimensions of keys g and g + 8 for
//     the scores and D / 8 contiguous dimensions of keys 2t, 2t+1, 2t+8, 2t+9
//     for the output: wide shared-memory loads, conflict-free under TMA's
//     128-byte swizzle at d = 128, and no transposition of V.  The weights go
//     from the score layout to the operand layout by movmatrix.
//   - Each of the four compute warps owns 16 keys of a 64-key tile with its own
//     running maxima, sums and output: no block-wide step per tile.  They are
//     joined in shared memory at the end of a segment piece.
// Work split: stream-K as in fa_decode.cuh, but over (batch entry, row block,
// 64-key tile) units without the head: the CTAs form groups of Hkv, a group
// takes a contiguous chunk of the units, and each of its CTAs does them for one
// key head.  A token's heads are neighbours in memory and a head's row is only
// d bytes, so a group's CTAs, walking the same tokens side by side, read whole
// DRAM pages between them; one head after the other, the same copies without
// any arithmetic streamed at 4.2 TB/s.  Partial records of shared segments are
// merged through their logsumexps by a second kernel.  Each CTA finds its chunk
// by scanning the lengths itself: no prefix launch.
//
// Measured, a call among others: 16 x 16(16) x 16384 x 128 full 190-205 us (1.08 GB:
// 0.81-0.87 of the copy bandwidth; the stream kernel alone 174 us under ncu),
// 64 x 32(8) x 8192 x 128 ragged and capped 109-121 us by the lengths drawn (0.54 GB
// on average: 0.68-0.76; the rest is the start, the piece ends and the merge), one
// 100-row cache 7 + 3 us on the device.  ncu: DRAM bytes within 3% of the algorithmic
// ones, issue slots 49% busy, tensor pipe 16%.
// More than 16 query rows read the cache again, 16 at a time, and at d = 128 the 168
// registers of NB = 2 do not hold queries, accumulators and values (280 to 360 bytes
// spilled): 16 sequences x 8 key heads x 16384 x 128, floor 83 us, take 102 us with 8
// rows per key head, 174 with 16, 326 with 32, 1197 with 128.
#pragma once
#include "fa_cache.cuh"
#include "fa_mod_fwd.cuh"

namespace fa {

// Stream CTAs: one wave.  NB = 1 fits three CTAs of 128 registers a thread on
// an SM, NB = 2 two of 168.
__host__ __device__ constexpr int cdec_ctas_per_sm(int NB) { return NB == 1 ? 3 : 2; }
constexpr int kCacheDecodeGroupsMax = 3 * 148;

struct CDecParams {
  const void* q;          // bf16 [B, Nq, H, d]
  void* o;                // bf16 [B, Nq, H, d]
  float* lse;             // [B, H, Nq]
  const uint8_t* kexp;    // [B, Hkv, Nk]
  const uint8_t* vexp;
  const int* seqlens;     // [B] or nullptr
  const float* slopes;    // [H] or nullptr
  int* bad;               // lengths outside the cache
  // {b, rb, 2 x first group + slot there, last group} of a segment that several
  // groups share, b = -1: not shared.  By segment b nrb + rb when there are no
  // more segments than groups, else by the group in whose chunk it ends (one at
  // most; the others end a segment they hold alone)
  int4* info;
  float* rec_o;           // [CTA][2][8 NB][d]
  float* rec_lse;         // [CTA][2][8 NB]
  int B, Nq, Nk, H, Hkv, G;
  int rows, nrb, rpb;     // G Nq query rows per key head, blocks of rpb = 8 NB
  int by_segment;
  int groups, causal, window;  // grid = groups * Hkv CTAs
  float scale_log2;       // scale log2 e          (no cap)
  float x_mul, cap_log2;  // scale / cap, cap log2 e
};

template <int D, int NB>
struct CDecCfg {
  static constexpr int KT = 64;
  static constexpr int NW = 4;                     // compute warps, 16 keys of a tile each
  static constexpr int R = 8 * NB;                 // query rows of a block
  static constexpr int TILE = KT * D;              // bytes of a K or V tile
  static constexpr int NSTAGE = (NB == 1 ? 4 : 6) * 128 / D;
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_ML = OFF_KV + NSTAGE * 2 * TILE;   // float [3][NW][R] m, mo, l
  static constexpr int OFF_ACC = OFF_ML + 3 * NW * R * 4;     // float [NW][4][D + 4]
  static constexpr int ACC_LD = D + 4;
  static constexpr int OFF_BAR = OFF_ACC + NW * 4 * ACC_LD * 4;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = NSTAGE, NBAR = 2 * NSTAGE;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  // misc: abort flag | per-warp ok [4]
  static constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;
  static constexpr int THREADS = 32 * (NW + 1);
  static constexpr int CTAS = cdec_ctas_per_sm(NB);
  static_assert(CTAS * (SMEM_BYTES + 1024) <= 233472, "CTAs per SM");
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
// transpose an 8 x 8 matrix of halves held two per lane (row lane / 4)
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int NB, bool CAP, bool BIAS>
__global__ void __launch_bounds__(160, cdec_ctas_per_sm(NB))
    fa_cache_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const CDecParams p) {
  using C = CDecCfg<D, NB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int n) -> uint32_t { return sbase + C::OFF_BAR + 8u * n; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  int* s_ok = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);  // [4] per compute warp

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NSTAGE; ++s) {
      mbar_init(bar(C::BAR_FULL + s), 1);
      mbar_init(bar(C::BAR_EMPTY + s), C::NW * 32);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::NW && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge waits for this grid's end itself

  // ---- this CTA's units: every warp scans the lengths for itself, each lane a
  // run of entries, so that no barrier stands before the first loads
  const int per = (p.B + 31) >> 5;
  const int e0 = min(p.B, lane * per), e1 = min(p.B, e0 + per);
  auto units = [&](int b) -> int {  // fits 32 bits: the host checks
    const int L = cdec_len(p, b);
    if (L < 0 || L > p.Nk) return -1;
    const CDecRange r = cdec_range(p, L);
    return (r.t1 - r.t0) * p.nrb;
  };
  long long sum = 0;
  bool bad = false;
#pragma unroll 4
  for (int b = e0; b < e1; ++b) {
    const int x = units(b);
    bad |= x < 0;
    sum += max(x, 0);
  }
  const bool any_bad = __any_sync(0xffffffffu, bad);
  long long inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += x;
  }
  const long long U = __shfl_sync(0xffffffffu, inc, 31);
  const long long chunk = (U + p.groups - 1) / p.groups;
  const int group = blockIdx.x / p.Hkv, hk = blockIdx.x % p.Hkv;  // hk: this CTA's key head
  const long long u0 = static_cast<long long>(group) * chunk;
  const long long u1 = min(U, u0 + chunk);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.bad = any_bad;
    if (any_bad) atomicOr(&g_fa_error_word, FA_DEVERR_BOUNDS);
  }
  if (any_bad || u0 >= u1) {  // lengths contradict the cache: write nothing; or no units (uniform over the CTA)
    if (!any_bad && !p.by_segment && hk == 0 && threadIdx.x == 0) p.info[group] = make_int4(-1, 0, 0, 0);
    return;
  }
  // the entry with unit u0, found by the lane whose run holds it
  int b0 = 0;
  long long base0 = inc - sum;
  const bool mine = base0 <= u0 && u0 < inc;
  if (mine) {
    b0 = e0;
    for (;;) {
      const int x = units(b0);
      if (u0 < base0 + x) break;
      base0 += x;
      ++b0;
    }
  }
  {
    const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    b0 = __shfl_sync(0xffffffffu, b0, from);
    base0 = __shfl_sync(0xffffffffu, base0, from);
  }
  __syncthreads();  // the barriers are set up

  // Walk of the units [u0, u1), the same in both roles: segment (b, rb),
  // its tiles [r.t0, r.t1), the current tile tp.
  struct Walk {
    int b, rb, tp, L;
    CDecRange r;
  };
  auto walk_begin = [&](Walk& w) {
    w.b = b0;
    w.L = cdec_len(p, w.b);
    w.r = cdec_range(p, w.L);
    const int rel = static_cast<int>(u0 - base0);
    const int T = w.r.t1 - w.r.t0;
    w.rb = rel / T;
    w.tp = w.r.t0 + rel % T;
  };
  auto walk_next = [&](Walk& w) {  // after the last tile of a segment, with units left
    if (++w.rb == p.nrb) {
      w.rb = 0;
      do {
        ++w.b;
        w.L = cdec_len(p, w.b);
        w.r = cdec_range(p, w.L);
      } while (w.r.t0 >= w.r.t1);
    }
    w.tp = w.r.t0;
  };

  if (warp == C::NW) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      Walk w;
      walk_begin(w);
      int issued = 0;
      bool ok = true;
      const int total = static_cast<int>(u1 - u0);
      // for the merge: the first segment, when it began before this chunk and ends in it
      const int before = w.tp - w.r.t0;
      const bool ends = w.r.t1 - w.tp <= total;
      int ended = 0;  // segments completed in this chunk; later ones are whole
      if (hk == 0) {
        int4 x = make_int4(-1, 0, 0, 0);
        if (before > 0 && ends) {
          const long long s0 = u0 - before;
          const int g0 = static_cast<int>(s0 / chunk);
          // group g0's piece is its last one (slot 1) unless its chunk starts with the
          // segment; every later group's piece is its first one (slot 0)
          x = make_int4(w.b, w.rb, 2 * g0 + (g0 * chunk < s0 ? 1 : 0), group);
        }
        if (!p.by_segment) p.info[group] = x;
        else if (ends) p.info[w.b * p.nrb + w.rb] = x;
      }
      for (int done = 0; ok && done < total; ++done) {
        const int st = issued % C::NSTAGE;
        if (!(ok = mbar_wait(bar(C::BAR_EMPTY + st), ((issued / C::NSTAGE) & 1) ^ 1u, abort_flag))) break;
        const int row = w.tp * C::KT;
        const int boxes = w.L - row > 32 ? 2 : 1;  // boxes of 32 keys; none past the length
        mbar_arrive_expect_tx(bar(C::BAR_FULL + st), boxes * 2 * 32 * D);
        const uint32_t dst = sbase + C::OFF_KV + st * 2 * C::TILE;
        for (int x = 0; x < boxes; ++x) {
          tma_load_4d(dst + x * 32 * D, &tmK, bar(C::BAR_FULL + st), 0, hk, row + 32 * x, w.b);
          tma_load_4d(dst + C::TILE + x * 32 * D, &tmV, bar(C::BAR_FULL + st), 0, hk, row + 32 * x, w.b);
        }
        ++issued;
        if (++w.tp == w.r.t1) {
          if (hk == 0 && p.by_segment && ended++ > 0) p.info[w.b * p.nrb + w.rb] = make_int4(-1, 0, 0, 0);
          if (done + 1 < total) walk_next(w);
        }
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
  constexpr int MT = D / 16;      // 16-dimension tiles of the output
  float* sMl = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* sAcc = reinterpret_cast<float*>(smem + C::OFF_ACC);
  constexpr float kLazy = 8.f;    // the maxima move when exceeded by more than 2^8
  const bool windowed = p.window > 0 && p.window < p.Nk;
  int gtile = 0;
  Walk w;
  walk_begin(w);
  const int total = static_cast<int>(u1 - u0);  // the host keeps a CTA's share below 2^31
  for (int done = 0; done < total;) {
    const int n = min(w.r.t1 - w.tp, total - done);
    const int L = w.L;
    // ---- query rows 8 nb + g of this row block: thread t takes D / 4
    // contiguous dimensions; scaled by 2^-a to below 2^15.  The scores come out
    // with rows 8 nb + 2t, 2t + 1 in this thread: row x = 2 nb + e below.
    uint32_t qb[NB][KS][2];
    float rowf[2 * NB], slope[2 * NB];
    int pos[2 * NB];               // the query's position
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = w.rb * C::R + 8 * nb + g;
      const bool row_ok = r < p.rows;
      const int qi = row_ok ? r / p.G : 0, h = hk * p.G + (row_ok ? r % p.G : 0);
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(p.q) + ((static_cast<size_t>(w.b) * p.Nq + qi) * p.H + h) * D + t * (D / 4));
      uint32_t x[D / 8];
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = row_ok ? src[i] : make_uint4(0u, 0u, 0u, 0u);
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
      const float rf = (CAP ? p.x_mul : p.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + ea) << 23);
      const float sl = BIAS ? slope_log2(p.slopes[h]) : 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {  // k-step s: this thread's dimensions 4s .. 4s + 3
        qb[nb][s][0] = pack_h2(bf16lo_to_f32(x[2 * s]) * mul, bf16hi_to_f32(x[2 * s]) * mul);
        qb[nb][s][1] = pack_h2(bf16lo_to_f32(x[2 * s + 1]) * mul, bf16hi_to_f32(x[2 * s + 1]) * mul);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = (2 * t + e) * 4;  // a lane that loaded row 2t + e
        rowf[2 * nb + e] = __shfl_sync(0xffffffffu, rf, from);
        slope[2 * nb + e] = BIAS ? __shfl_sync(0xffffffffu, sl, from) : 0.f;
        pos[2 * nb + e] = L - p.Nq + __shfl_sync(0xffffffffu, qi, from);
      }
    }
    float m[2 * NB], mo[2 * NB], l[2 * NB];
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
      m[x] = mo[x] = -INFINITY;
      l[x] = 0.f;
    }
    float acc[MT][NB][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[i][nb][0] = acc[i][nb][1] = acc[i][nb][2] = acc[i][nb][3] = 0.f;

    // keys [key_lo, L) are those that some query of the entry sees
    const int key_lo = windowed ? max(0, L - p.Nq - p.window + 1) : 0;
    // exponent bytes of this thread's keys g, g + 8 (keys, values), fetched one tile
    // ahead.  With a cap, a key no query sees gets a key scale of (minus) 0, whatever it
    // holds: its score is 0 where the form of the tanh is chosen.  (Zeroing the scores
    // there instead, or two comparisons a key here, costs 1 to 2% of a capped call.)
    const size_t plane = (static_cast<size_t>(w.b) * p.Hkv + hk) * p.Nk + warp * 16 + g;
    const uint8_t *ke = p.kexp + plane, *ve = p.vexp + plane;
    const uint32_t span = static_cast<uint32_t>(L - key_lo);
    uint32_t ex[4];
    auto fetch_exp = [&](int tile) {
      const int k = tile * C::KT;
      if constexpr (CAP) {
        const uint32_t at = static_cast<uint32_t>(k + warp * 16 + g - key_lo);
        ex[0] = at < span ? ke[k] : 256u;  // e8m0_value: -0
        ex[1] = at + 8u < span ? ke[k + 8] : 256u;
        ex[2] = at < span ? ve[k] : 127u;
        ex[3] = at + 8u < span ? ve[k + 8] : 127u;
      } else {
        const int left = L - warp * 16 - g - k;
        ex[0] = left > 0 ? ke[k] : 127u;
        ex[1] = left > 8 ? ke[k + 8] : 127u;
        ex[2] = left > 0 ? ve[k] : 127u;
        ex[3] = left > 8 ? ve[k + 8] : 127u;
      }
    };
    fetch_exp(w.tp);
    // keys that all queries of the entry see
    const int full_lo = windowed ? L - p.window : 0;
    const int full_hi = min(p.causal ? L - p.Nq + 1 : L, windowed ? L - p.Nq + p.window : L);
    bool ok = true;
    for (int it = 0; it < n; ++it, ++gtile) {
      const int st = gtile % C::NSTAGE;
      const int k0 = (w.tp + it) * C::KT + warp * 16;  // this warp's first key
      // score factor and value exponent of keys g and g + 8
      const float ks[2] = {e8m0_value(ex[0]), e8m0_value(ex[1])};
      const float ev[2] = {ex[2] == 255u ? __uint_as_float(0x7fffffffu) : static_cast<float>(ex[2]) - 127.f,
                           ex[3] == 255u ? __uint_as_float(0x7fffffffu) : static_cast<float>(ex[3]) - 127.f};
      if (it + 1 < n) fetch_exp(w.tp + it + 1);
      ok = mbar_wait(bar(C::BAR_FULL + st), (gtile / C::NSTAGE) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint8_t* pK = smem + C::OFF_KV + st * 2 * C::TILE + warp * 16 * D;
      const uint8_t* pV = pK + C::TILE;
      if (k0 < L) {  // warp-uniform
        // ---- scores: keys g and g + 8
        uint32_t kw[2][KS];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = 8 * x + g;
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            // 16-byte chunk (D / 64) t + i of the row, swizzled as TMA wrote it
            const int ch = (D == 128) ? ((2 * t + i) ^ (r & 7)) : (t ^ ((r >> 1) & 3));
            const uint4 v = *reinterpret_cast<const uint4*>(pK + r * D + ch * 16);
            kw[x][4 * i] = v.x;
            kw[x][4 * i + 1] = v.y;
            kw[x][4 * i + 2] = v.z;
            kw[x][4 * i + 3] = v.w;
          }
        }
        float sc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sc[nb][0] = sc[nb][1] = sc[nb][2] = sc[nb][3] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_h2(kw[0][s], a0, a2);
          e4m3x4_to_h2(kw[1][s], a1, a3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_f16(sc[nb], a0, a1, a2, a3, qb[nb][s][0], qb[nb][s][1]);
        }
        // the values' loads, ahead of the softmax arithmetic: keys 2t, 2t+1 (first half of k) and 2t+8, 2t+9
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
        // ---- z in base 2 and exponents of the weights, zo = z + ev.  Element c:
        // key g + 8 (c >> 1), row x = 2 nb + (c & 1).  A key that a row does not
        // see is a select, so that its scale (NaN perhaps) stays out.
        const bool all_see = k0 >= full_lo && k0 + 16 <= full_hi;  // warp-uniform
        float so[NB][4];
        bool over = false;
        uint64_t z2[NB][2];  // (row 2t, row 2t + 1) of keys g and g + 8
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            z2[nb][e] = fmul2(f2_pack(sc[nb][2 * e], sc[nb][2 * e + 1]),
                              f2_pack(rowf[2 * nb] * ks[e], rowf[2 * nb + 1] * ks[e]));
        if constexpr (CAP) {
          // the polynomial within its range: the exponential form's error is
          // 6e-8 of the cap even where the scores are small
          float ax = 0.f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float a, b;
              f2_unpack(z2[nb][e], a, b);
              ax = fmax3(ax, fabsf(a), fabsf(b));
            }
          const uint64_t cl2 = f2_pack(p.cap_log2, p.cap_log2);
          if (__all_sync(0xffffffffu, ax <= kTanhRange)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 2; ++e) z2[nb][e] = fmul2(tanh2_poly(z2[nb][e]), cl2);
          } else {
            const uint64_t xe2 = f2_pack(kTwoLog2e, kTwoLog2e), cm2 = f2_pack(-2.f * p.cap_log2, -2.f * p.cap_log2);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 2; ++e) z2[nb][e] = tanh2_any(fmul2(z2[nb][e], xe2), cl2, cm2);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          f2_unpack(z2[nb][0], sc[nb][0], sc[nb][1]);
          f2_unpack(z2[nb][1], sc[nb][2], sc[nb][3]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int x = 2 * nb + (c & 1), key = k0 + g + 8 * (c >> 1);
            float z = sc[nb][c];
            if (BIAS) z = fmaf(-slope[x], fabsf(static_cast<float>(pos[x] - key)), z);
            float zo = z + ev[c >> 1];
            if (!all_see) {
              const int away = pos[x] - key;
              const bool see = key < L && (!p.causal || away >= 0) &&
                               (p.window <= 0 || (away < p.window && -away < p.window));
              z = see ? z : -INFINITY;
              zo = see ? zo : -INFINITY;
            }
            sc[nb][c] = z;
            so[nb][c] = zo;
            over |= z > m[x] + kLazy || zo > mo[x] + kLazy;
          }
        if (__any_sync(0xffffffffu, over)) {  // some maximum moves: reduce it over the keys' lanes
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int x = 2 * nb + e;
              float a = fmaxf(sc[nb][e], sc[nb][2 + e]), b = fmaxf(so[nb][e], so[nb][2 + e]);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
              }
              if (a > m[x]) {
                l[x] *= ex2(m[x] - a);
                m[x] = a;
              }
              if (b > mo[x]) {
                const float f = ex2(mo[x] - b);
                mo[x] = b;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  acc[i][nb][e] *= f;
                  acc[i][nb][2 + e] *= f;
                }
              }
            }
        }
        // ---- weights, from (key, row pair) to (row, key pair) lanes
        uint32_t wb[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float nm[2], nmo[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = 2 * nb + e;
            nm[e] = m[x] == -INFINITY ? 0.f : m[x];
            nmo[e] = mo[x] == -INFINITY ? 0.f : mo[x];
            l[x] += ex2(sc[nb][e] - nm[e]) + ex2(sc[nb][2 + e] - nm[e]);
          }
          wb[nb][0] = movmatrix_trans(pack_h2(ex2(so[nb][0] - nmo[0]), ex2(so[nb][1] - nmo[1])));
          wb[nb][1] = movmatrix_trans(pack_h2(ex2(so[nb][2] - nmo[0]), ex2(so[nb][3] - nmo[1])));
        }
        // ---- output
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
        for (int c = 0; c < D / 32; ++c) {  // four dimensions, two output tiles at a time
          // bytes (key, key + 1) of dimensions 4c .. 4c + 3 of the thread's chunk
          const uint32_t a01 = __byte_perm(vw[0][c], vw[1][c], 0x5140), a23 = __byte_perm(vw[0][c], vw[1][c], 0x7362);
          const uint32_t b01 = __byte_perm(vw[2][c], vw[3][c], 0x5140), b23 = __byte_perm(vw[2][c], vw[3][c], 0x7362);
          uint32_t h0, h1, h2, h3, i0, i1, i2, i3;
          e4m3x4_to_h2(a01, h0, h1);
          e4m3x4_to_h2(b01, h2, h3);
          e4m3x4_to_h2(a23, i0, i1);
          e4m3x4_to_h2(b23, i2, i3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma_f16(acc[2 * c][nb], h0, h1, h2, h3, wb[nb][0], wb[nb][1]);
            mma_f16(acc[2 * c + 1][nb], i0, i1, i2, i3, wb[nb][0], wb[nb][1]);
          }
        }
      }
      mbar_arrive(bar(C::BAR_EMPTY + st));
    }
    // ---- join the four warps: rows of the block in passes of four
    if (lane == 0) s_ok[warp] = ok;
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], off);
      if (g == 0) {
        const int row = 8 * (x >> 1) + 2 * t + (x & 1);
        sMl[(0 * C::NW + warp) * C::R + row] = m[x];
        sMl[(1 * C::NW + warp) * C::R + row] = mo[x];
        sMl[(2 * C::NW + warp) * C::R + row] = l[x];
      }
    }
    named_bar_sync(1, C::NW * 32);
    // a wait gave up in some warp: the error word is set; write nothing more
    // (every warp reads the same four flags, so all of them leave)
    if (!(s_ok[0] && s_ok[1] && s_ok[2] && s_ok[3])) return;
    const bool whole = w.tp == w.r.t0 && n == w.r.t1 - w.r.t0;  // the piece is the whole segment
    const int slot = done == 0 ? 0 : 1;
    const int nrows = min(C::R, p.rows - w.rb * C::R);
    // rows 4 x4 .. 4 x4 + 3 at a time: lanes t = 2 (x4 & 1), + 1.  Not unrolled:
    // this runs once or twice a CTA, where fetching its instructions costs more
    // than the selects (four copies of it took 9 us of a 31 us call)
#pragma unroll 1
    for (int r0 = 0; r0 < nrows; r0 += 4) {
      const bool hi = NB == 2 && r0 >= 8;
      if ((t >> 1) == ((r0 >> 2) & 1)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = (r0 & 8) + 2 * t + e;
          const float mow = hi ? mo[2 * (NB - 1) + e] : mo[e];
          float M = -INFINITY;
#pragma unroll
          for (int y = 0; y < C::NW; ++y) M = fmaxf(M, sMl[(C::NW + y) * C::R + row]);
          // this warp's output factor: 2^(mo_w - mo), 0 when it saw nothing
          const float f = mow == -INFINITY ? 0.f : ex2(mow - M);
          float* dst = sAcc + (warp * 4 + (row & 3)) * C::ACC_LD + g * (D / 8);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            *reinterpret_cast<float2*>(dst + 2 * i) = make_float2((hi ? acc[i][NB - 1][e] : acc[i][0][e]) * f,
                                                                  (hi ? acc[i][NB - 1][2 + e] : acc[i][0][2 + e]) * f);
        }
      }
      named_bar_sync(1, C::NW * 32);
      const int row = r0 + warp;  // warp = row of the pass
      if (row < nrows) {
        float M = -INFINITY, MO = -INFINITY, lsum = 0.f;
#pragma unroll
        for (int y = 0; y < C::NW; ++y) {
          M = fmaxf(M, sMl[y * C::R + row]);
          MO = fmaxf(MO, sMl[(C::NW + y) * C::R + row]);
        }
#pragma unroll
        for (int y = 0; y < C::NW; ++y) {
          const float mw = sMl[y * C::R + row], lw = sMl[(2 * C::NW + y) * C::R + row];
          // a warp without a maximum has seen nothing (l = 0) or NaN only (l = NaN)
          lsum += mw == -INFINITY ? lw : lw * ex2(mw - M);
        }
        const float inv = lsum == 0.f ? 0.f : __fdividef(ex2(MO - M), lsum);
        const float lse = lsum == 0.f ? -INFINITY : (M + lg2(lsum)) * kLn2;
        const int r = w.rb * C::R + row, qi = r / p.G, h = hk * p.G + r % p.G;
        const size_t rec = (static_cast<size_t>(blockIdx.x) * 2 + slot) * C::R + row;
        constexpr int PL = D / 32;  // columns per lane, PL at a time
        float a[PL];
#pragma unroll
        for (int c = 0; c < PL; ++c) a[c] = 0.f;
#pragma unroll
        for (int y = 0; y < C::NW; ++y)
#pragma unroll
          for (int c = 0; c < PL; c += 2) {
            const float2 v = *reinterpret_cast<const float2*>(sAcc + (y * 4 + warp) * C::ACC_LD + lane * PL + c);
            a[c] += v.x;
            a[c + 1] += v.y;
          }
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) +
                             ((static_cast<size_t>(w.b) * p.Nq + qi) * p.H + h) * D + lane * PL;
#pragma unroll
        for (int c = 0; c < PL; c += 2) {
          if (whole) *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(a[c] * inv, a[c + 1] * inv);
          else *reinterpret_cast<float2*>(p.rec_o + rec * D + lane * PL + c) = make_float2(a[c] * inv, a[c + 1] * inv);
        }
        if (lane == 0) {
          float* dst = whole ? p.lse + (static_cast<size_t>(w.b) * p.H + h) * p.Nq + qi : p.rec_lse + rec;
          *dst = lse;
        }
      }
      named_bar_sync(1, C::NW * 32);
    }
    done += n;
    w.tp += n;
    if (w.tp == w.r.t1 && done < total) walk_next(w);
  }
}

// Merge of the records of segments that several groups share: one block per
// (segment, key head; row), or, where there are more segments than groups, per
// (group, key head; row) for the one such segment that may end in its chunk.
// The block's warps take the records in turn, eight in flight each, under a
// maximum of their own, and join at the end.  The blocks also write O = 0,
// LSE = -inf for entries whose queries see no tile.  Bound by the latency of
// three dependent loads and by the launch of its blocks (per group always, the
// 4736 blocks of 148 records shared by two segments took 16 us; four rows a
// block 14 us).
template <int D>
__global__ void __launch_bounds__(512) fa_cache_decode_merge_kernel(const CDecParams p) {
  __shared__ float s_m[16], s_den[16];
  __shared__ float s_acc[16][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the stream kernel has ended and its writes are visible
  const int idx = blockIdx.x / p.Hkv, hk = blockIdx.x % p.Hkv;
  const int4 seg = p.info[idx];
  if (*p.bad) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int r_in = blockIdx.y;  // row of the row block
  if (p.by_segment) {
    const int b = idx / p.nrb, r = (idx % p.nrb) * p.rpb + r_in;
    const CDecRange rg = cdec_range(p, cdec_len(p, b));
    if (rg.t0 >= rg.t1) {  // nobody wrote info for this segment
      if (r < p.rows) {
        const int qi = r / p.G, h = hk * p.G + r % p.G;
        uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) +
                                                  ((static_cast<size_t>(b) * p.Nq + qi) * p.H + h) * D);
        if (threadIdx.x < D / 2) o[threadIdx.x] = 0u;
        if (threadIdx.x == 0) p.lse[(static_cast<size_t>(b) * p.H + h) * p.Nq + qi] = -INFINITY;
      }
      return;
    }
  } else if (hk == 0 && r_in == 0) {
#pragma unroll 1
    for (int b = idx; b < p.B; b += p.groups) {
      const CDecRange rg = cdec_range(p, cdec_len(p, b));
      if (rg.t0 < rg.t1) continue;
      const int64_t rows = static_cast<int64_t>(p.Nq) * p.H;
      uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + b * rows * D);
#pragma unroll 1
      for (int64_t i = threadIdx.x; i < rows * D / 2; i += blockDim.x) o[i] = 0u;
#pragma unroll 1
      for (int64_t i = threadIdx.x; i < rows; i += blockDim.x) p.lse[b * rows + i] = -INFINITY;
    }
  }
  const int r = seg.y * p.rpb + r_in;    // row of its key head
  if (seg.x < 0 || r >= p.rows) return;  // uniform over the block
  const int g0 = seg.z >> 1, slot0 = seg.z & 1, n = seg.w - g0 + 1;
  constexpr int PL = D / 32;  // columns per lane
  constexpr float kLog2ef = 1.4426950408889634f;
  float m = -INFINITY, den = 0.f, acc[PL];
#pragma unroll
  for (int c = 0; c < PL; ++c) acc[c] = 0.f;
#pragma unroll 1
  for (int k0 = warp; k0 < n; k0 += 8 * nw) {
    float ls[8], v[8][PL];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + nw * i;
      ls[i] = -INFINITY;
#pragma unroll
      for (int c = 0; c < PL; ++c) v[i][c] = 0.f;
      if (k < n) {
        const size_t cta = static_cast<size_t>(g0 + k) * p.Hkv + hk;
        const size_t rec = (cta * 2 + (k == 0 ? slot0 : 0)) * p.rpb + r_in;
        ls[i] = p.rec_lse[rec] * kLog2ef;
        const float* o = p.rec_o + rec * D + lane * PL;
        if constexpr (PL == 4) {
          const float4 x = *reinterpret_cast<const float4*>(o);
          v[i][0] = x.x;
          v[i][1] = x.y;
          v[i][2] = x.z;
          v[i][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(o);
          v[i][0] = x.x;
          v[i][1] = x.y;
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) mn = fmaxf(mn, ls[i]);
    const float ref = mn == -INFINITY ? 0.f : mn;  // no weight yet: all 0 (or NaN)
    const float al = m == -INFINITY ? 1.f : ex2(m - ref);
    m = mn;
    den *= al;
#pragma unroll
    for (int c = 0; c < PL; ++c) acc[c] *= al;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float wk = ex2(ls[i] - ref);
      den += wk;
#pragma unroll
      for (int c = 0; c < PL; ++c) acc[c] = fmaf(wk, v[i][c], acc[c]);
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_den[warp] = den;
  }
#pragma unroll
  for (int c = 0; c < PL; ++c) s_acc[warp][lane * PL + c] = acc[c];
  __syncthreads();
  if (warp > 0) return;
  float mx = -INFINITY;
#pragma unroll 4
  for (int y = 0; y < nw; ++y) mx = fmaxf(mx, s_m[y]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  den = 0.f;
#pragma unroll
  for (int c = 0; c < PL; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int y = 0; y < nw; ++y) {
    // a share without a maximum has weight 0, or NaN sums that stay NaN
    const float f = s_m[y] == -INFINITY ? 1.f : ex2(s_m[y] - ref);
    den = fmaf(f, s_den[y], den);
#pragma unroll
    for (int c = 0; c < PL; ++c) acc[c] = fmaf(f, s_acc[y][lane * PL + c], acc[c]);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int qi = r / p.G, h = hk * p.G + r % p.G;
  __nv_bfloat16* out =
      static_cast<__nv_bfloat16*>(p.o) + ((static_cast<size_t>(seg.x) * p.Nq + qi) * p.H + h) * D + lane * PL;
#pragma unroll
  for (int c = 0; c < PL; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0)
    p.lse[(static_cast<size_t>(seg.x) * p.H + h) * p.Nq + qi] = den == 0.f ? -INFINITY : (ref + lg2(den)) * kLn2;
}

}  // namespace fa
