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
// Both kernels are bound by HBM (append: 2d read, d + 1 written per row; read:
// d + 1 read, 2d written), a handful of instructions per 8 values.
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
// 2^(e - 127) for an exponent byte (E8M0: 255 is NaN, 0 is 2^-127)
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
  int tb;                 // tokens per block
};

// One block per (token chunk, batch entry); blockIdx.z: keys or values.  A row
// takes D / 8 lanes of 16 bytes.
template <int D>
__global__ void __launch_bounds__(256) fa_cache_append_kernel(const CacheAppendParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int b = blockIdx.y, z = blockIdx.z;
  const int start = p.start[b];
  const int count = p.count ? p.count[b] : p.T;
  if (count < 0 || count > p.T || start < 0 || start > p.Nk - count) {  // does not fit: report, write nothing
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_fa_error_word, FA_DEVERR_BOUNDS);
    return;
  }
  const int t0 = blockIdx.x * p.tb;
  const int nrow = (min(count, t0 + p.tb) - t0) * p.Hkv;  // rows (token, head) of this block
  const int lane = threadIdx.x & 31, sub = lane / LPR, part = lane % LPR;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(z ? p.v : p.k) +
                             (static_cast<size_t>(b) * p.T + t0) * p.Hkv * D;
  uint8_t* codes = (z ? p.vcodes : p.kcodes) + (static_cast<size_t>(b) * p.Nk + start + t0) * p.Hkv * D;
  uint8_t* exps = (z ? p.vexp : p.kexp) + static_cast<size_t>(b) * p.Hkv * p.Nk + start + t0;
  constexpr int U = 4, STEP = 8 * RPW;  // rows per block step
  for (int r0 = (threadIdx.x >> 5) * RPW + sub; r0 - sub < nrow; r0 += U * STEP) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nrow) v[u] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<size_t>(r) * D + part * 8));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      float x[8], a = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo_to_f32(w[i]);
        x[2 * i + 1] = bf16hi_to_f32(w[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x[i]);
        a = fmaxf(a, m < INFINITY ? m : 0.f);  // NaN and infinities left out
      }
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
      const uint32_t e = e8m0_of_amax(a);
      const float inv = __uint_as_float((254u - e) << 23);  // 2^(127 - e), exact
      if (e == 247u) {  // a row with values from 1.75 2^127 on
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (fabsf(x[i]) < INFINITY) x[i] = fminf(fmaxf(x[i], -1.875f * 0x1p127f), 1.875f * 0x1p127f);
      }
      const uint32_t lo = pack_e4m3x2_sat(x[0] * inv, x[1] * inv) | pack_e4m3x2_sat(x[2] * inv, x[3] * inv) << 16;
      const uint32_t hi = pack_e4m3x2_sat(x[4] * inv, x[5] * inv) | pack_e4m3x2_sat(x[6] * inv, x[7] * inv) << 16;
      if (r < nrow) {
        *reinterpret_cast<uint2*>(codes + static_cast<size_t>(r) * D + part * 8) = make_uint2(lo, hi);
        if (part == 0) exps[static_cast<size_t>(r % p.Hkv) * p.Nk + r / p.Hkv] = static_cast<uint8_t>(e);
      }
    }
  }
}

struct CacheReadParams {
  const uint8_t* codes;  // [B, Nk, Hkv, d]
  const uint8_t* exps;   // [B, Hkv, Nk]
  const int* seqlens;    // [B] or nullptr (Nk)
  void* out;             // bf16 [B, Nk, Hkv, d]
  int Nk, Hkv, tb;
};

// One block per (token chunk, batch entry).  Rows at or past the entry's length
// are written as zero and their cache rows are not read.
template <int D>
__global__ void __launch_bounds__(256) fa_cache_read_kernel(const CacheReadParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int b = blockIdx.y;
  const int L = p.seqlens ? p.seqlens[b] : p.Nk;
  if (L < 0 || L > p.Nk) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_fa_error_word, FA_DEVERR_BOUNDS);
    return;
  }
  const int t0 = blockIdx.x * p.tb;
  const int nrow = (min(p.Nk, t0 + p.tb) - t0) * p.Hkv;
  const int nread = max(0, min(L, t0 + p.tb) - t0) * p.Hkv;
  const int lane = threadIdx.x & 31, sub = lane / LPR, part = lane % LPR;
  const size_t base = (static_cast<size_t>(b) * p.Nk + t0) * p.Hkv * D;
  const uint8_t* codes = p.codes + base;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + base;
  const uint8_t* exps = p.exps + static_cast<size_t>(b) * p.Hkv * p.Nk + t0;
  constexpr int U = 4, STEP = 8 * RPW;
  for (int r0 = (threadIdx.x >> 5) * RPW + sub; r0 < nrow; r0 += U * STEP) {
    uint2 v[U];
    uint32_t e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      v[u] = make_uint2(0u, 0u);
      e[u] = 127u;
      if (r < nread) {
        v[u] = __ldcs(reinterpret_cast<const uint2*>(codes + static_cast<size_t>(r) * D + part * 8));
        e[u] = exps[static_cast<size_t>(r % p.Hkv) * p.Nk + r / p.Hkv];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * STEP;
      const float sc = e8m0_value(e[u]);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t h = e4m3x2_to_h2((i < 2 ? v[u].x : v[u].y) >> (16 * (i & 1)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        w[i] = pack_bf16x2(f.x * sc, f.y * sc);
      }
      if (r < nrow)
        *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * D + part * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace fa
