// Mask plan of the modified-score attention: which keys each query sees, as
// one interval per query.
//
// Causality, a sliding window, packed documents and a visible prefix all leave
// query i a contiguous run of keys, lo_i <= j < hi_i:
//     documents   [first, last + 1) of the run of equal ids around i;
//                 a negative id is padding: the row sees nothing
//     causal      hi_i <= max(i + 1, prefix_b)
//     window W    lo_i >= i - W + 1, hi_i <= i + W
// so a plan is two integers per query (not an N x N mask), and per 128-row
// tile the range of tiles of the other side that it meets, which is what the
// attention kernels loop over.  The plan depends on the batch alone and is
// made once for all layers, heads and directions.
//
// One block per 1024 rows, a thread a row.  The run of equal ids around a row
// comes from a scan over the block; a run that reaches past the block is followed
// outside it, 4096 ids at a time.  The ranges of query tiles per key tile need
// the tiles of the whole entry: a second small kernel, or the same block where
// there is only one.  Bound by latency (one block per entry took 22 us at
// N = 16384, three per cent of the attention that uses the plan).
#pragma once
#include "sm100_ptx.cuh"

namespace fa {

// Per 128-query tile: key tiles [kbeg, kend) hold every key any of its rows
// sees; keys in [full_lo, full_hi) are seen by all of its rows; `ahead` is 1
// when some row sees a key after itself (it decides on which side of the
// diagonal a distance bias can be taken as linear).
struct __align__(16) PlanQTile {
  int kbeg, kend, full_lo, full_hi;
  int ahead, pad[3];
};
// Per 128-key tile: query tiles [qbeg, qend) hold every query that sees any of
// its keys.
struct PlanKTile {
  int qbeg, qend;
};

struct PlanView {
  int2* rows;       // [B, N] {lo, hi}; {0, 0} for a row that sees nothing
  PlanQTile* qt;    // [B, T], T = ceil(N / 128)
  PlanKTile* kt;    // [B, T]
};

constexpr int kPlanThreads = 1024;

// Query tiles that meet key tile k: first and last overlap (tiles in between
// that do not overlap are masked row by row).  A warp per key tile.
__device__ __forceinline__ void plan_ktile(const PlanView& pv, size_t b, int T, int k) {
  const PlanQTile* qt = pv.qt + b * T;
  int q0 = T, q1 = 0;
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < T; i += 32) {
    const int2 r = *reinterpret_cast<const int2*>(qt + i);  // kbeg, kend
    if (r.x <= k && k < r.y) {
      q0 = min(q0, i);
      q1 = i + 1;
    }
  }
  q0 = __reduce_min_sync(0xffffffffu, q0);
  q1 = __reduce_max_sync(0xffffffffu, q1);
  if ((threadIdx.x & 31) == 0) {
    PlanKTile t;
    t.qbeg = q1 > 0 ? q0 : 0;
    t.qend = q1;
    pv.kt[b * T + k] = t;
  }
}

__global__ void __launch_bounds__(kPlanThreads)
    fa_mask_plan_kernel(PlanView pv, const int* __restrict__ doc_ids, const int* __restrict__ prefix_len, int N,
                        int window, int causal) {
  __shared__ int s_a[32], s_b[32];
  __shared__ int s_tile[8][5];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the tile kernel waits for this grid itself
  const int b = blockIdx.y, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int T = (N + 127) >> 7;
  const int base = blockIdx.x * kPlanThreads, end = min(N, base + kPlanThreads);
  const int i = base + t;  // this thread's row
  if (t < 8) {
    s_tile[t][0] = s_tile[t][3] = N;  // min lo, min hi
    s_tile[t][1] = s_tile[t][2] = s_tile[t][4] = 0;  // max hi, max lo, ahead
  }
  int lo = 0, hi = N;
  bool pad = false;
  if (doc_ids) {
    const int* ids = doc_ids + static_cast<size_t>(b) * N;
    auto is_start = [&](int k) { return k == 0 || ids[k] != ids[k - 1]; };
    const bool start = i < N && is_start(i);
    pad = i < N && ids[i] < 0;
    // last start at or before this row, first start after it, within the block
    int mx = start ? i : -1, mn = start ? i : N;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, mx, off), y = __shfl_down_sync(0xffffffffu, mn, off);
      if (lane >= off) mx = max(mx, x);
      if (lane < 32 - off) mn = min(mn, y);
    }
    if (lane == 31) s_a[warp] = mx;
    if (lane == 0) s_b[warp] = mn;
    mn = __shfl_down_sync(0xffffffffu, mn, 1);
    if (lane == 31) mn = N;
    __syncthreads();
    for (int w = 0; w < warp; ++w) mx = max(mx, s_a[w]);
    for (int w = warp + 1; w < 32; ++w) mn = min(mn, s_b[w]);
    __syncthreads();
    // the start of the run that reaches into the block from before it
    int before = base;
    if (!is_start(base)) {  // uniform; base > 0
      int found = -1;
      for (int k1 = base; found < 0 && k1 > 0; k1 -= 4 * kPlanThreads) {  // position 0 is a start
        int f = -1;
        for (int e = 0; e < 4; ++e) {
          const int k = k1 - 4 * kPlanThreads + 4 * t + e;
          if (k >= 0 && k < k1 && is_start(k)) f = k;
        }
        f = __reduce_max_sync(0xffffffffu, f);
        if (lane == 0) s_a[warp] = f;
        __syncthreads();
        for (int w = 0; w < 32; ++w) found = max(found, s_a[w]);
        __syncthreads();
      }
      before = found;
    }
    // and the first start behind the block
    int after = N;
    for (int k0 = end; after == N && k0 < N; k0 += 4 * kPlanThreads) {
      int f = N;
      for (int e = 3; e >= 0; --e) {
        const int k = k0 + 4 * t + e;
        if (k < N && is_start(k)) f = k;
      }
      f = __reduce_min_sync(0xffffffffu, f);
      if (lane == 0) s_b[warp] = f;
      __syncthreads();
      for (int w = 0; w < 32; ++w) after = min(after, s_b[w]);
      __syncthreads();
    }
    lo = mx >= 0 ? mx : before;
    hi = mn < N ? mn : after;
  } else {
    __syncthreads();  // s_tile is set
  }
  if (i < N) {
    if (causal) {
      const int pre = prefix_len ? min(max(prefix_len[b], 0), N) : 0;
      hi = min(hi, max(i + 1, pre));
    }
    if (window > 0) {
      lo = max(lo, i - window + 1);
      hi = min(hi, window < N ? i + window : N);
    }
    if (pad || lo >= hi) lo = hi = 0;
    pv.rows[static_cast<size_t>(b) * N + i] = make_int2(lo, hi);
  } else {
    lo = hi = 0;
  }
  // tile ranges: a warp's rows lie in one tile
  {
    const bool in = i < N, some = in && lo < hi;
    const int lo_min = __reduce_min_sync(0xffffffffu, some ? lo : N);
    const int hi_max = __reduce_max_sync(0xffffffffu, some ? hi : 0);
    const int lo_max = __reduce_max_sync(0xffffffffu, in ? lo : 0);
    const int hi_min = __reduce_min_sync(0xffffffffu, in ? hi : N);
    const int ahead = __any_sync(0xffffffffu, some && hi > i + 1);
    if (lane == 0) {
      int* x = s_tile[warp >> 2];
      atomicMin(x + 0, lo_min);
      atomicMax(x + 1, hi_max);
      atomicMax(x + 2, lo_max);
      atomicMin(x + 3, hi_min);
      atomicOr(x + 4, ahead);
    }
  }
  __syncthreads();
  PlanQTile* qt = pv.qt + static_cast<size_t>(b) * T;
  const int k = blockIdx.x * 8 + t;
  if (t < 8 && k < T) {
    const int* x = s_tile[t];
    PlanQTile q;
    q.kbeg = x[1] > 0 ? x[0] >> 7 : 0;
    q.kend = x[1] > 0 ? (x[1] + 127) >> 7 : 0;
    q.full_lo = x[2];
    q.full_hi = x[3];
    q.ahead = x[4];
    q.pad[0] = q.pad[1] = q.pad[2] = 0;
    qt[k] = q;
  }
  if (gridDim.x == 1) {
    __syncthreads();  // the block's tiles are visible to the block
    if (warp < T) plan_ktile(pv, b, T, warp);
  }
}

__global__ void __launch_bounds__(128) fa_mask_plan_tiles_kernel(PlanView pv, int T) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' kernel has ended and its tiles are visible
  const int k = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (k < T) plan_ktile(pv, blockIdx.y, T, k);
}

}  // namespace fa
