// append_e2m1.cu -- the rows of an append into a 4-bit pool (KV_DTYPE_E2M1),
// behind the plan kernel of append.cu: kv_append_quantize, kv_append_from_pool
// and the append of kv_decode_step.
//
// "Smaller, faster, safer: running Kimi and GLM at scale", section "Quantizing
// the KV cache": half the bytes, twice the resident context; here half of the
// e4m3 pool's again (9/16 with the group scales).
//
// One warp per (page, kv head, K|V) tile, its rows in registers (e2m1.cuh).
// Bounded by HBM for prompts: 2 bytes a value in, 9/16 out.
#include <climits>

#include "append_items.cuh"
#include "common.cuh"
#include "e2m1.cuh"
#include "internal.h"

namespace kvfp8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtas = 3;  // resident CTAs an SM of the bulk kernel

// Tiles t0, t0 + kWarps, .. (even: K of head t / 2, odd: V) of request r's
// logical page jp, by this warp.
template <bool FROM_POOL>
__device__ __forceinline__ void page_tiles(const AppendArgs& a, int r, long long n, long long Lnew,
                                           long long jp, int t0, int t1) {
  const kv_pool_desc& d = a.d;
  const long long L0 = Lnew - n, H = d.num_kv_heads;
  const long long lo = max(jp * 16, L0), hi = min((jp + 1) * 16, Lnew);
  const int nrows = (int)(hi - lo), slot0 = (int)(lo - jp * 16);
  const int p = a.page_table[(long long)r * a.max_pages + jp];
  const int sp = FROM_POOL ? a.src_page_table[(long long)r * a.src_max_pages + jp] : 0;
  if (p < 0 || p >= d.num_pages || (FROM_POOL && (sp < 0 || sp >= a.src.num_pages))) {
    if ((threadIdx.x & 31) == 0) set_error(d.ctl, KV_ERR_BAD_PAGE_ID);
    return;
  }
  const bool fresh = jp * 16 >= L0;  // popped by this call
  // a partly filled page that this call's pops handed to a later request is
  // not written through the stale mapping
  if (!fresh && d.tags[p] != a.exp_tags[(long long)r * a.max_pages + jp]) return;
  const long long row0 = FROM_POOL ? 0 : a.new_indptr[r] + (lo - L0);
  for (int t = t0; t < t1; t += kWarps) {
    const long long h = t >> 1, tile = p * H + h;
    uint8_t* kc = static_cast<uint8_t*>(d.k_cache) + tile * kE2m1Tile;
    uint8_t* vc = static_cast<uint8_t*>(d.v_cache) + tile * kE2m1Tile;
    if ((t & 1) == 0) {
      if (FROM_POOL)
        e2m1_k_tile(static_cast<const uint16_t*>(a.src.k_cache) + (sp * H + h) * 2048, 128, nrows,
                    0, true, d.k_scale + tile, kc);
      else
        e2m1_k_tile(a.k_new + (row0 * H + h) * 128, H * 128, nrows, slot0, fresh, d.k_scale + tile,
                    kc);
    } else {
      if (FROM_POOL)
        e2m1_v_tile_dim_major(static_cast<const uint16_t*>(a.src.v_cache) + (sp * H + h) * 2048,
                              nrows, d.v_scale + tile, vc);
      else
        e2m1_v_tile(a.v_new + (row0 * H + h) * 128, H * 128, nrows, slot0, fresh,
                    d.v_scale + tile, vc);
    }
  }
}

// Few rows a request: a CTA per (request, touched page, 8 tiles).
__global__ void __launch_bounds__(kThreads) append_e2m1_rows_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  if (r >= a.d.ctl[KV_CTL_APPEND_STOP]) return;
  const long long n = req_rows(a, r), Lnew = a.seq_lens[r];
  const int t0 = blockIdx.z * kWarps + (threadIdx.x >> 5);
  if (n <= 0 || t0 >= 2 * a.d.num_kv_heads) return;
  for (long long jp = (Lnew - n) / 16 + blockIdx.y; jp * 16 < Lnew; jp += gridDim.y)
    page_tiles<false>(a, r, n, Lnew, jp, t0, min(t0 + 1, 2 * a.d.num_kv_heads));
}

// Many rows: persistent CTAs, each taking whole pages in turn.
template <bool FROM_POOL>
__global__ void __launch_bounds__(kThreads, kCtas) append_e2m1_bulk_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int pre[];
  __shared__ int wsum[kWarps];
  const int B = min(a.B, (int)a.d.ctl[KV_CTL_APPEND_STOP]);
  const int total = B > 0 ? bulk_items_prefix(a, B, 1, pre, wsum) : 0;
  __syncthreads();
  for (int it = blockIdx.x; it < total; it += gridDim.x) {
    const int r = item_owner(pre, B, it);
    const long long n = req_rows(a, r), Lnew = a.seq_lens[r];
    page_tiles<FROM_POOL>(a, r, n, Lnew, (Lnew - n) / 16 + (it - pre[r]), threadIdx.x >> 5,
                          2 * a.d.num_kv_heads);
  }
}

}  // namespace

cudaError_t launch_append_e2m1(const AppendArgs& a, long long pages, cudaStream_t s,
                               int* launches) {
  const int sms = sm_count();
  const bool bulk = (a.from_pool || a.max_new >= 32) && sms > 0 && a.B <= kMaxPersistB &&
                    (long long)a.B * pages <= INT_MAX;
  if (a.from_pool && !bulk) return cudaErrorNotSupported;
  cudaError_t e;
  if (bulk) {
    const auto kernel = a.from_pool ? append_e2m1_bulk_kernel<true> : append_e2m1_bulk_kernel<false>;
    const size_t smem = sizeof(int) * ((size_t)a.B + 1);
    if (smem > 40 * 1024) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(kernel, dim3((unsigned)sms * kCtas), dim3(kThreads), smem, s, a);
  } else {
    const unsigned z = (2u * a.d.num_kv_heads + kWarps - 1) / kWarps;
    if (z > 65535) return cudaErrorInvalidConfiguration;
    e = launch_pdl(append_e2m1_rows_kernel, dim3((unsigned)a.B, (unsigned)min(pages, 65535LL), z),
                   dim3(kThreads), 0, s, a);
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
