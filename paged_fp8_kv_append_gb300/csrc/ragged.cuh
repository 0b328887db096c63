// ragged.cuh -- work items of a ragged batch without a prefix pass.
//
// Request r of a batch has the flat rows indptr[r] .. indptr[r+1]-1, which lie
// in consecutive pages of its own from any slot on.  n rows touch at most
// floor((n - 2) / P) + 2 pages, and
//   first(r) = floor(indptr[r] / P) + 2 r
// leaves floor(indptr[r+1] / P) - floor(indptr[r] / P) + 2 >= floor(n / P) + 2
// item numbers to request r: enough for every page it touches, at most two a
// request left over.  An item finds its request by searching indptr alone, so
// a kernel over a batch's pages needs neither a plan launch nor a scan.
#pragma once

#include "common.cuh"

namespace kvfp8 {

__host__ __device__ inline long long ragged_items(long long total_rows, int B, int P) {
  return total_rows / P + 2LL * B;
}

__device__ __forceinline__ long long ragged_first(long long row, int P, int r) {
  return row / P + 2LL * r;
}

// The request whose item numbers hold `item`, found by a whole warp: 32 entries a step.
// Always in [0, B).  Only the first `limit` requests are looked at (their rows must not run
// backwards; what is behind them may), though the loads do not wait for it.
__device__ __forceinline__ int ragged_owner(const int32_t* indptr, int B, int limit, int P,
                                            long long item) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool in = lane * step < n;
    const int32_t row = in ? indptr[at] : 0;
    const bool le = in && (lane == 0 || (at < limit && ragged_first(row, P, at) <= item));
    const int k = 31 - __clz((int)__ballot_sync(0xffffffffu, le));
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// The same by reading the offsets in order, 128 a step: -1 where no request's items begin at or
// before `item`, and only requests before the first whose rows run backwards.  (A search does
// not see such a place.)
__device__ __forceinline__ int ragged_owner_in_order(const int32_t* indptr, int B, int P,
                                                     long long item) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  int owner = -1;
  bool more = true;
  for (int base = 0; more && base < B; base += 32 * kAhead) {
    int32_t i0[kAhead], i1[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = base + 32 * k + lane;
      i0[k] = r < B ? indptr[r] : 0;
      i1[k] = r < B ? indptr[r + 1] : 0;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = base + 32 * k + lane;
      const uint32_t back = __ballot_sync(0xffffffffu, i1[k] < i0[k]);
      const uint32_t le =
          __ballot_sync(0xffffffffu, r < B && ragged_first(i0[k], P, r) <= item) &
          (back != 0 ? (back & (0u - back)) - 1u : 0xffffffffu);
      if (more) owner += __popc(le);
      more = more && le == 0xffffffffu;
    }
  }
  return owner;
}

}  // namespace kvfp8
