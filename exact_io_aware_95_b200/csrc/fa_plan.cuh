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
// One block per batch entry.  The runs of equal ids come from two block scans
// (last start at or before i, first start after i) over per-thread chunks; the
// tile ranges from warp reductions over 128 rows.  Bound by latency: about
// 6 us at N = 16384, against hundreds of microseconds for the attention that
// uses it.
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

__global__ void __launch_bounds__(kPlanThreads)
    fa_mask_plan_kernel(PlanView pv, const int* __restrict__ doc_ids, const int* __restrict__ prefix_len, int N,
                        int window, int causal) {
  __shared__ int s_last[32], s_first[32];
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int T = (N + 127) >> 7;
  int2* rows = pv.rows + static_cast<size_t>(b) * N;
  const int pre = prefix_len ? min(max(prefix_len[b], 0), N) : 0;
  auto finish = [&](int i, int lo, int hi) {
    if (causal) hi = min(hi, max(i + 1, pre));
    if (window > 0) {
      lo = max(lo, i - window + 1);
      hi = min(hi, window < N ? i + window : N);
    }
    if (lo >= hi) lo = hi = 0;
    rows[i] = make_int2(lo, hi);
  };
  if (!doc_ids) {
    for (int i = t; i < N; i += kPlanThreads) finish(i, 0, N);
  } else {
    const int* ids = doc_ids + static_cast<size_t>(b) * N;
    const int per = (N + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(N, t * per), i1 = min(N, i0 + per);
    // this thread's chunk: its last and its first run start
    int last = -1, first = N;
    int prev = i0 > 0 && i0 < N ? ids[i0 - 1] : 0;
    for (int i = i0; i < i1; ++i) {
      const int id = ids[i];
      if (i == 0 || id != prev) {
        last = i;
        if (first == N) first = i;
      }
      prev = id;
    }
    // exclusive scans over the threads: maximum of `last` from the left,
    // minimum of `first` from the right
    int mx = last, mn = first;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, mx, off), c = __shfl_down_sync(0xffffffffu, mn, off);
      if (lane >= off) mx = max(mx, a);
      if (lane < 32 - off) mn = min(mn, c);
    }
    if (lane == 31) s_last[warp] = mx;
    if (lane == 0) s_first[warp] = mn;
    __syncthreads();
    int left = __shfl_up_sync(0xffffffffu, mx, 1), right = __shfl_down_sync(0xffffffffu, mn, 1);
    if (lane == 0) left = -1;
    if (lane == 31) right = N;
    for (int w = 0; w < warp; ++w) left = max(left, s_last[w]);
    for (int w = warp + 1; w < kPlanThreads / 32; ++w) right = min(right, s_first[w]);
    // walk the chunk backwards for the run ends, run by run
    int end = right;
    for (int i = i1; i > i0;) {
      // the run that holds row i - 1 inside this chunk starts at s
      int s = i - 1;
      while (s > i0 && ids[s - 1] == ids[s]) --s;
      int lo = s;
      if (s == i0 && !(i0 == 0 || ids[i0 - 1] != ids[i0])) lo = left;  // it began before the chunk
      const bool pad = ids[s] < 0;
      for (int r = s; r < i; ++r) {
        if (pad) rows[r] = make_int2(0, 0);
        else finish(r, lo, end);
      }
      end = s;
      i = s;
    }
  }
  __syncthreads();  // the block's rows are visible to the block
  // tile ranges: one warp per query tile
  PlanQTile* qt = pv.qt + static_cast<size_t>(b) * T;
  for (int k = warp; k < T; k += kPlanThreads / 32) {
    int lo_min = N, hi_max = 0, lo_max = 0, hi_min = N, ahead = 0;
    for (int r = lane; r < 128; r += 32) {
      const int i = 128 * k + r;
      if (i < N) {
        const int2 x = rows[i];
        lo_max = max(lo_max, x.x);
        hi_min = min(hi_min, x.y);
        if (x.x < x.y) {
          lo_min = min(lo_min, x.x);
          hi_max = max(hi_max, x.y);
          ahead |= x.y > i + 1;
        }
      }
    }
    lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    hi_max = __reduce_max_sync(0xffffffffu, hi_max);
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    ahead = __any_sync(0xffffffffu, ahead);
    if (lane == 0) {
      PlanQTile q;
      q.kbeg = hi_max > 0 ? lo_min >> 7 : 0;
      q.kend = hi_max > 0 ? (hi_max + 127) >> 7 : 0;
      q.full_lo = lo_max;
      q.full_hi = hi_min;
      q.ahead = ahead;
      q.pad[0] = q.pad[1] = q.pad[2] = 0;
      qt[k] = q;
    }
  }
  __syncthreads();
  // query tiles that meet each key tile: first and last overlap (tiles in
  // between that do not overlap are masked row by row)
  PlanKTile* kt = pv.kt + static_cast<size_t>(b) * T;
  for (int k = t; k < T; k += kPlanThreads) {
    int q0 = T, q1 = 0;
    for (int i = 0; i < T; ++i) {
      if (qt[i].kbeg <= k && k < qt[i].kend) {
        q0 = min(q0, i);
        q1 = i + 1;
      }
    }
    kt[k].qbeg = q1 > 0 ? q0 : 0;
    kt[k].qend = q1;
  }
}

}  // namespace fa
