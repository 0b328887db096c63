// append_items.cuh -- the work items of a bulk append, shared by the append
// kernels of e4m3 and bf16 pools (append.cu) and of 4-bit ones (append_e2m1.cu).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace kvfp8 {

// Rows request r appends in this call (none when the step mask drops it).
__device__ __forceinline__ long long req_rows(const AppendArgs& a, int r) {
  if (a.step_mask != nullptr && a.step_mask[r] != 0) return 0;
  if (a.from_pool) return a.src_lens[r];
  return (long long)a.new_indptr[r + 1] - a.new_indptr[r];
}

// Work items of a bulk append: every (request, page this call touches),
// times per_page (tiles per page for GQA, 1 for latent), in request order.
// The CTA's threads build the inclusive prefix pre[0..B] in shared memory, so
// a persistent grid visits only real work however few requests have rows.
constexpr int kMaxPersistB = 16384;

static __device__ int bulk_items_prefix(const AppendArgs& a, int B, int per_page, int* pre, int* wsum) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const long long P = a.d.page_size;
  int carry = 0;
  if (threadIdx.x == 0) pre[0] = 0;
  for (int base = 0; base < B; base += blockDim.x) {
    const int r = base + threadIdx.x;
    int v = 0;
    if (r < B) {
      const long long n = req_rows(a, r);
      if (n > 0) {
        const long long Lnew = a.seq_lens[r], L0 = Lnew - n;
        v = (int)((Lnew - 1) / P - L0 / P + 1) * per_page;
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) wsum[wid] = v;
    __syncthreads();
    int before = carry;
    for (int k = 0; k < wid; ++k) before += wsum[k];
    if (r < B) pre[r + 1] = before + v;
    int chunk = 0;
    for (int k = 0; k < nw; ++k) chunk += wsum[k];
    carry += chunk;
    __syncthreads();
  }
  return carry;
}

// request owning item i: the r with pre[r] <= i < pre[r + 1]
__device__ __forceinline__ int item_owner(const int* pre, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace kvfp8
