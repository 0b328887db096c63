// append_e2m1.cu -- the rows of an append into a 4-bit pool (KV_DTYPE_E2M1),
// behind the plan kernel of append.cu: kv_append_quantize, kv_append_from_pool
// and the append of kv_decode_step.
//
// "Smaller, faster, safer: running Kimi and GLM at scale", section "Quantizing
// the KV cache": half the bytes, twice the resident context; here half of the
// e4m3 pool's again (9/16 with the group scales).
//
// One warp per (page, kv head, K|V) tile (e2m1.cuh).  Bounded by HBM for
// prompts and handoffs: 2 bytes a value in, 9/16 out.  There a warp takes its tiles through
// a ring of its own in shared memory: its lanes copy a tile's rows
// asynchronously, 16 bytes each and neighbours together, and read them back in
// the order that the tile's layout wants.  Straight from global memory that
// order costs half sectors (row-major) or words 512 bytes apart (a bf16
// pool's dim-major V): the L1 was busy 85% at 5.1 TB/s.
//   handoff of 16 requests of 4k-32k tokens, 8 heads: 205 us, 5.9 TB/s (190 in this
//     kernel at 6.4, of the 6.8 of a plain copy; its pages are popped here too, on all
//     SMs: one by one in the plan's block they took 25 us)
//   8 prompts of 1k-4k tokens: 31 us, of which the plan 9 and this kernel 18 (5.3 TB/s)
//   a row of 64 requests: 8 us of plan and 6 of the rows' kernel, dependent loads
#include <climits>

#include "append_items.cuh"
#include "common.cuh"
#include "e2m1.cuh"
#include "internal.h"

namespace kvfp8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// ------------------------------------------------- few rows a request

// A CTA per (request, touched page, 8 tiles).
__global__ void __launch_bounds__(kThreads) append_e2m1_rows_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const kv_pool_desc& d = a.d;
  const int r = blockIdx.x, t = blockIdx.z * kWarps + (threadIdx.x >> 5);  // tile: 2 head + K|V
  const long long H = d.num_kv_heads, h = t >> 1;
  if (r >= d.ctl[KV_CTL_APPEND_STOP]) return;
  const long long n = req_rows(a, r), Lnew = a.seq_lens[r], L0 = Lnew - n;
  if (n <= 0 || t >= 2 * H) return;
  for (long long jp = L0 / 16 + blockIdx.y; jp * 16 < Lnew; jp += gridDim.y) {
    const long long lo = max(jp * 16, L0), hi = min((jp + 1) * 16, Lnew);
    const int nrows = (int)(hi - lo), slot0 = (int)(lo - jp * 16);
    const int p = a.page_table[(long long)r * a.max_pages + jp];
    if (p < 0 || p >= d.num_pages) {
      if ((threadIdx.x & 31) == 0) set_error(d.ctl, KV_ERR_BAD_PAGE_ID);
      continue;
    }
    const bool fresh = jp * 16 >= L0;  // popped by this call
    // a partly filled page that this call's pops handed to a later request is
    // not written through the stale mapping
    if (!fresh && d.tags[p] != a.exp_tags[(long long)r * a.max_pages + jp]) continue;
    const long long row0 = a.new_indptr[r] + (lo - L0), tile = p * H + h;
    if ((t & 1) == 0)
      e2m1_k_tile<false>(GlobalRows{a.k_new + (row0 * H + h) * 128, H * 128}, nrows, slot0, fresh,
                         d.k_scale + tile, static_cast<uint8_t*>(d.k_cache) + tile * kE2m1Tile);
    else
      e2m1_v_tile<false>(GlobalRows{a.v_new + (row0 * H + h) * 128, H * 128}, nrows, slot0, fresh,
                         d.v_scale + tile, static_cast<uint8_t*>(d.v_cache) + tile * kE2m1Tile);
  }
}

// ------------------------------------------------- many rows

constexpr int kStages = 3, kCtas = 2;     // tiles in a warp's ring; CTAs an SM
constexpr int kTileBytes = 16 * 128 * 2;  // a tile's bf16 rows

// A tile to quantise.
struct Item {
  const uint16_t* src;
  int tile;       // (page, kv head); -1: nothing to do
  uint8_t nrows, slot0, fresh, is_v;
};
static_assert(sizeof(Item) == 16, "one shared load");

__device__ __forceinline__ void copy16(uint32_t dst_smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst_smem), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Where a tile's 16-byte chunks lie in its stage, so that the eight lanes of a load's
// phase read eight different banks of 16 bytes.
//   K rows of 16 chunks: a phase reads chunks 2t of two neighbouring rows
__device__ __forceinline__ int k_chunk(int row, int c) { return 16 * row + (c ^ (row & 1)); }
//   V rows: a phase reads two chunks, 2 apart, of rows 0, 2, 4, 6 (+ a constant)
__device__ __forceinline__ int v_chunk(int row, int c) {
  return 16 * row + (c ^ ((row >> 1 & 1) | (row & 4)));
}
//   dim-major V, two chunks a dim: 4-byte loads of 8 dims 16 apart
__device__ __forceinline__ int d_chunk(int q) { return q ^ (q >> 5 & 7); }

template <bool FROM_POOL>
__global__ void __launch_bounds__(kThreads, kCtas) append_e2m1_bulk_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int wsum[kWarps];
  const kv_pool_desc& d = a.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Item* items = reinterpret_cast<Item*>(smem + kWarps * kStages * kTileBytes) + warp * 64;
  int* pre = reinterpret_cast<int*>(smem + kWarps * (kStages * kTileBytes + 64 * (int)sizeof(Item)));
  const int B = min(a.B, (int)d.ctl[KV_CTL_APPEND_STOP]);
  const int pages = B > 0 ? bulk_items_prefix(a, B, 1, pre, wsum) : 0;
  __syncthreads();
  const long long head0 = (long long)d.ctl[KV_CTL_FREE_HEAD] - pages;  // of a handoff's pops
  const uint32_t ring = smem_u32(smem) + warp * (kStages * kTileBytes);
  const int H = d.num_kv_heads;
  const long long tiles = 2LL * H * pages, step = (long long)gridDim.x * kWarps;
  const long long first = (long long)blockIdx.x * kWarps + warp;
  // this warp's tiles: i = 0, 1, .. are first + step i
  const int count = first < tiles ? (int)((tiles - first + step - 1) / step) : 0;

  // items 32 b .. of the table, one a lane
  auto fill = [&](int b) {
    Item m{nullptr, -1, 0, 0, 0, 0};
    const int i = 32 * b + lane;
    if (i < count) {
      const long long x = first + step * i;
      const int page = (int)(x / (2 * H)), t = (int)(x - (long long)page * 2 * H), h = t >> 1;
      const int r = item_owner(pre, B, page);
      const long long n = req_rows(a, r), Lnew = a.seq_lens[r], L0 = Lnew - n;
      const long long jp = L0 / 16 + (page - pre[r]);
      const long long lo = max(jp * 16, L0), hi = min((jp + 1) * 16, Lnew);
      const long long row0 = FROM_POOL ? 0 : a.new_indptr[r] + (lo - L0);
      const long long at = (long long)r * a.max_pages + jp;
      // a handoff's pages are popped here (a.defer_pops): every request was empty, so the
      // touched pages, in order, are the popped ones
      const int p = FROM_POOL ? d.free_list[head0 + page] : a.page_table[at];
      const int sp = FROM_POOL ? a.src_page_table[(long long)r * a.src_max_pages + jp] : 0;
      m.fresh = jp * 16 >= L0;  // popped by this call
      m.is_v = t & 1;
      m.nrows = (uint8_t)(hi - lo);
      m.slot0 = (uint8_t)(lo - jp * 16);
      if (FROM_POOL)
        m.src = static_cast<const uint16_t*>(m.is_v ? a.src.v_cache : a.src.k_cache) +
                ((long long)sp * H + h) * 2048;
      else
        m.src = (m.is_v ? a.v_new : a.k_new) + (row0 * H + h) * 128;
      if (FROM_POOL && t == 0 && p >= 0 && p < d.num_pages) {  // (each page once)
        const uint32_t tag = d.tags[p] + 1u;  // wraps mod 2^32
        d.tags[p] = tag;
        a.page_table[at] = p;
        a.exp_tags[at] = tag;
      }
      if (p < 0 || p >= d.num_pages || (FROM_POOL && (sp < 0 || sp >= a.src.num_pages)))
        set_error(d.ctl, KV_ERR_BAD_PAGE_ID);
      // a partly filled page that this call's pops handed to a later request is
      // not written through the stale mapping
      else if (m.fresh || d.tags[p] == a.exp_tags[at])
        m.tile = p * H + h;  // (2^31 tiles are 2 TB)
    }
    items[32 * (b & 1) + lane] = m;
    __syncwarp();
  };
  auto fetch = [&](int i, int st) {
    if (i < count) {
      const Item m = items[i & 63];
      const uint32_t dst = ring + st * kTileBytes;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(m.src);
      if (m.tile >= 0) {
        if (FROM_POOL && m.is_v) {  // (the whole tile: it lies in the page)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            copy16(dst + 16 * d_chunk(lane + 32 * k), src + 16 * (lane + 32 * k));
        } else {
          const long long stride = FROM_POOL ? 256 : 256LL * H;
          const int c = lane & 15;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = 2 * k + (lane >> 4);
            if (row < m.nrows)
              copy16(dst + 16 * (m.is_v ? v_chunk(row, c) : k_chunk(row, c)),
                     src + row * stride + 16 * c);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (count > 0) fill(0);
  if (count > 32) fill(1);
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) fetch(i, i);
  int st = 0;
  for (int i = 0; i < count; ++i) {
    if ((i & 31) == 0 && i > 0 && i + 32 < count) fill((i >> 5) + 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const Item m = items[i & 63];
    const uint32_t at = ring + st * kTileBytes;
    if (m.tile >= 0) {
      uint8_t* cache = static_cast<uint8_t*>(m.is_v ? d.v_cache : d.k_cache);
      uint8_t* dst = cache + (long long)m.tile * kE2m1Tile;
      float* scale = (m.is_v ? d.v_scale : d.k_scale) + m.tile;
      auto k_row = [&](int row, int c) { return lds128(at + 16 * k_chunk(row, c)); };
      auto v_row = [&](int row, int c) { return lds128(at + 16 * v_chunk(row, c)); };
      auto v_dim = [&](int dd, int w) { return lds32(at + 16 * d_chunk(2 * dd + (w >> 2)) + 4 * (w & 3)); };
      if (!m.is_v) {
        if (m.nrows == 16)
          e2m1_k_tile<true>(k_row, 16, 0, true, scale, dst);
        else
          e2m1_k_tile<false>(k_row, m.nrows, m.slot0, m.fresh, scale, dst);
      } else if (FROM_POOL) {
        if (m.nrows == 16)
          e2m1_v_tile_dim_major<true>(v_dim, 16, scale, dst);
        else
          e2m1_v_tile_dim_major<false>(v_dim, m.nrows, scale, dst);
      } else {
        if (m.nrows == 16)
          e2m1_v_tile<true>(v_row, 16, 0, true, scale, dst);
        else
          e2m1_v_tile<false>(v_row, m.nrows, m.slot0, m.fresh, scale, dst);
      }
    }
    __syncwarp();  // every lane has read its part of the stage
    fetch(i + kStages, st);
    if (++st == kStages) st = 0;
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
    const auto kernel =
        a.from_pool ? append_e2m1_bulk_kernel<true> : append_e2m1_bulk_kernel<false>;
    constexpr size_t kFixed = kWarps * (kStages * kTileBytes + 64 * sizeof(Item));
    const size_t smem = kFixed + sizeof(int) * ((size_t)a.B + 1);
    // (the largest batch's: the same from every thread that may be between this and its launch)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kFixed + sizeof(int) * (kMaxPersistB + 1)));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3((unsigned)sms * kCtas), dim3(kThreads), smem, s, a);
  } else {
    const unsigned z = (2u * a.d.num_kv_heads + kWarps - 1) / kWarps;
    e = launch_pdl(append_e2m1_rows_kernel, dim3((unsigned)a.B, (unsigned)min(pages, 65535LL), z),
                   dim3(kThreads), 0, s, a);
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
