// 8-bit key/value cache: quantising rows as they are written, reading them back.
//
// A row (one token of one key head, d values) is stored as d e4m3 codes and one
// exponent byte e (the OCP E8M0 form, value 2^(e - 127)):
//     e    = the smallest with amax <= 448 2^(e - 127), at least 1
//     code = e4m3(x 2^(127 - e)), round to nearest even, saturating
// amax is taken over the row's finite values; NaN stays NaN, an infinity
// becomes +-448 2^(e - 127), and a row without a finite non-zero value gets
// e = 127.  Finite values beyond +-1.875 2^127 are taken as that: the code above
// would stand for 2^128, an infinity in bf16.  The scale is a power of two, so it costs no rounding of its own:
// quantising is one rounding (relative error at most 2^-4, or half a step of
// 2^(e - 127 - 9) at the row's small end), and reading back is exact in bf16
// (four significant bits times a power of two).
//
// Caches are [B, Nk, Hkv, d] bytes, exponents [B, Hkv, Nk] so that the keys of
// one head are contiguous where the decoding kernel streams them.
//
// Reading is bound by HBM (d + 1 bytes read and 2d written per row): 8 x 8191 x 8 x
// 128 half full in 28.4-29.6 us (168 MB: 0.87-0.90 of the copy bandwidth).  Appending
// (2d read, d + 1 written) is bound by instruction issue as much: 8 x 2047 x 8 x 128
// in 16.7 us of device time (76 MB: 0.69), 72% of the issue slots busy.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sm100_ptx.cuh"

namespace fa {

// two e4m3 codes (low 16 bits) -> two halves, exact
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t codes) {
  uint32_t r;
  const unsigned short c = static_cast<unsigned short>(codes);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// the four codes of a word -> halves (codes 0, 1) and (codes 2, 3); the 16-bit
// halves of the word are named, not shifted out
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t& h01, uint32_t& h23) {
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(h01), "=r"(h23)
      : "r"(w));
}
// two floats -> two e4m3 codes, `lo` in the low byte; saturating, NaN stays NaN
__device__ __forceinline__ uint32_t pack_e4m3x2_sat(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^(e - 127) for an exponent byte (E8M0: 255 is NaN, 0 is 2^-127); -0 for 256
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fffffffu : (e == 0u ? 0x00400000u : e << 23));
}
// exponent byte of a row whose largest finite magnitude is amax
__device__ __forceinline__ uint32_t e8m0_of_amax(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  if (bits == 0u) return 127u;
  // amax = 1.f 2^(E - 127): 448 = 1.75 2^8, so 2^(E - 127 - 8) suffices up to 1.75
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return e < 1 ? 1u : static_cast<uint32_t>(e);
}

struct CacheAppendParams {
  const void *k, *v;        // bf16 [B, T, Hkv, d]
  uint8_t *kcodes, *vcodes; // [B, Nk, Hkv, d]
  uint8_t *kexp, *vexp;     // [B, Hkv, Nk]
  const int* start;       // [B] first row written
  const int* count;       // [B] rows written, or nullptr (T)
  int T, Nk, Hkv;
  int tb, hb, hchunks;      // a block: tb tokens of all heads, or one token of hb heads
};

// One block per (token chunk, batch entry); blockIdx.z: keys or values.  A row
// takes D / 8 lanes of 16 bytes.  Bound by instruction issue as much as by HBM,
// so the usual row costs as few as possible: the maximum is taken of packed
// bf16 magnitudes; rows with an infinity, a NaN maximum or values from 1.75 2^127
// on leave for a slow path, voted on by warp; the exponent bytes are collected
// in shared memory and written head by head.  8 x 2047 x 8 x 128 (half to all of
// it valid): 21.6 -> 16.5 us.
constexpr int kCacheRows = 256;  // rows (token, head) of a block at most; the host's split keeps to it

template <int D>
__global__ void __launch_bounds__(256) fa_cache_append_kernel(const CacheAppendParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  __shared__ uint8_t s_e[kCacheRows];
  const int b = blockIdx.y, z = blockIdx.z;
  const int start = p.start[b];
  const int count = p.count ? p.count[b] : p.T;
  if (count < 0 || count > p.T || start < 0 || start > p.Nk - count) {  // does not fit: report, write nothing
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_fa_error_word, FA_DEVERR_BOUNDS);
    return;
  }
  // rows r0 + c0 .. of this block: a token chunk, and a part of the heads where
  // one token has more than fit
  const int t0 = blockIdx.x / p.hchunks * p.tb, h0 = blockIdx.x % p.hchunks * p.hb;
  const int nt = min(count, t0 + p.tb) - t0, nh = min(p.Hkv - h0, p.hb);
  if (nt <= 0) return;  // uniform over the block
  const int nrow = nt * nh;  // contiguous: either all heads of the tokens, or one token
  const int lane = threadIdx.x & 31, sub = lane / LPR, part = lane % LPR;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(z ? p.v : p.k) +
                             ((static_cast<size_t>(b) * p.T + t0) * p.Hkv + h0) * D + part * 8;
  uint8_t* codes = (z ? p.vcodes : p.kcodes) +
                   ((static_cast<size_t>(b) * p.Nk + start + t0) * p.Hkv + h0) * D + part * 8;
  constexpr int U = 4, STEP = 8 * RPW;  // rows per block step
  for (int r0 = (threadIdx.x >> 5) * RPW + sub; r0 - sub < nrow; r0 += U * STEP) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nrow) v[u] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<size_t>(r) * D));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      // largest magnitude of the row, both halves of a word at a time (the
      // packed maximum passes over NaN unless both are)
      auto mag = [](uint32_t x) {
        x &= 0x7fff7fffu;
        return *reinterpret_cast<const __nv_bfloat162*>(&x);
      };
      __nv_bfloat162 m2 = __hmax2(__hmax2(mag(w[0]), mag(w[1])), __hmax2(mag(w[2]), mag(w[3])));
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&m2), off);
        m2 = __hmax2(m2, *reinterpret_cast<const __nv_bfloat162*>(&o));
      }
      const uint32_t mw = *reinterpret_cast<const uint32_t*>(&m2);
      uint32_t top = max(mw & 0xffffu, mw >> 16);  // bits of the row's maximum, as bf16
      uint64_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = f2_pack(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i]));
      if (__any_sync(0xffffffffu, top >= 0x7f60u)) {  // an infinity, NaN or values from 1.75 2^127 on
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y[2];
          f2_unpack(x[i], y[0], y[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (fabsf(y[c]) < INFINITY) {
              y[c] = fminf(fmaxf(y[c], -1.875f * 0x1p127f), 1.875f * 0x1p127f);
              a = fmaxf(a, fabsf(y[c]));
            }
          x[i] = f2_pack(y[0], y[1]);
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        top = __float_as_uint(a) >> 16;
      }
      const uint32_t e = e8m0_of_amax(__uint_as_float(top << 16));
      const float inv = __uint_as_float((254u - e) << 23);  // 2^(127 - e), exact
      const uint64_t inv2 = f2_pack(inv, inv);
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y0, y1;
        f2_unpack(fmul2(x[i], inv2), y0, y1);
        c[i] = pack_e4m3x2_sat(y0, y1);
      }
      if (r < nrow) {
        *reinterpret_cast<uint2*>(codes + static_cast<size_t>(r) * D) =
            make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
        if (part == 0) s_e[r] = static_cast<uint8_t>(e);
      }
    }
  }
  __syncthreads();
  uint8_t* exps = (z ? p.vexp : p.kexp) + (static_cast<size_t>(b) * p.Hkv + h0) * p.Nk + start + t0;
  for (int i = threadIdx.x; i < nrow; i += 256) {
    const int h = i / nt, t = i - h * nt;
    exps[static_cast<size_t>(h) * p.Nk + t] = s_e[t * nh + h];
  }
}

struct CacheReadParams {
  const uint8_t* codes;  // [B, Nk, Hkv, d]
  const uint8_t* exps;   // [B, Hkv, Nk]
  const int* seqlens;    // [B] or nullptr (Nk)
  void* out;             // bf16 [B, Nk, Hkv, d]
  int Nk, Hkv;
  int tb, hb, hchunks;
};

// One block per (token chunk, batch entry).  Rows at or past the entry's length
// are written as zero and their cache rows are not read.  The exponent bytes
// come through shared memory, read head by head.
template <int D>
__global__ void __launch_bounds__(256) fa_cache_read_kernel(const CacheReadParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  __shared__ float s_sc[kCacheRows];
  const int b = blockIdx.y;
  const int L = p.seqlens ? p.seqlens[b] : p.Nk;
  if (L < 0 || L > p.Nk) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_fa_error_word, FA_DEVERR_BOUNDS);
    return;
  }
  const int t0 = blockIdx.x / p.hchunks * p.tb, h0 = blockIdx.x % p.hchunks * p.hb;
  const int nt = min(p.Nk, t0 + p.tb) - t0, nh = min(p.Hkv - h0, p.hb);
  const int nrow = nt * nh;                        // contiguous, as in the append
  const int ntr = max(0, min(L, t0 + p.tb) - t0), nread = ntr * nh;
  const int lane = threadIdx.x & 31, sub = lane / LPR, part = lane % LPR;
  const size_t base = ((static_cast<size_t>(b) * p.Nk + t0) * p.Hkv + h0) * D + part * 8;
  const uint8_t* codes = p.codes + base;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + base;
  const uint8_t* exps = p.exps + (static_cast<size_t>(b) * p.Hkv + h0) * p.Nk + t0;
  for (int i = threadIdx.x; i < nread; i += 256) {
    const int h = i / ntr, t = i - h * ntr;
    s_sc[t * nh + h] = e8m0_value(exps[static_cast<size_t>(h) * p.Nk + t]);
  }
  constexpr int U = 4, STEP = 8 * RPW;
  const int first = (threadIdx.x >> 5) * RPW + sub;
  uint2 v[U];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      v[u] = make_uint2(0u, 0u);
      if (r < nread) v[u] = __ldcs(reinterpret_cast<const uint2*>(codes + static_cast<size_t>(r) * D));
    }
  };
  load(first);
  __syncthreads();
  for (int r0 = first; r0 < nrow; r0 += U * STEP) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      const float sc = r < nread ? s_sc[r] : 0.f;
      const uint64_t sc2 = f2_pack(sc, sc);
      uint32_t h[4], w[4];
      e4m3x4_to_h2(v[u].x, h[0], h[1]);
      e4m3x4_to_h2(v[u].y, h[2], h[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        float y0, y1;
        f2_unpack(fmul2(f2_pack(f.x, f.y), sc2), y0, y1);
        w[i] = pack_bf16x2(y0, y1);
      }
      if (r < nrow)
        *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * D) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    load(r0 + U * STEP);
  }
}

}  // namespace fa
