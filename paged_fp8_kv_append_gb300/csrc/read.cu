// read.cu -- kv_read_rows: cached rows back as contiguous bf16 rows.
//
// "Smaller, faster, safer: running Kimi and GLM at scale", section
// "Quantizing the KV cache": prefill works on a bf16 cache and decode on an
// e4m3 one.  Rows that leave the pool (to a bf16 prefill that reuses a prefix,
// to another worker) are x = bf16(code * scale), one multiplication in fp32
// and one rounding; bf16 pools copy the bits.
//
// Bounded by HBM: per row width codes in, 2 * width bytes out.  One CTA per
// touched page: a page's tiles are contiguous, so every load and store of a
// warp is a run of whole sectors; V tiles (dim-major) are transposed in
// registers, a lane holding 4 dims of all 16 tokens.
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"
#include "ragged.cuh"

namespace kvfp8 {
namespace {

constexpr int kThreads = 256;

// bf16(code * scale) of the two codes in the low half of w, packed
__device__ __forceinline__ uint32_t dequant2(uint32_t w, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
  return *reinterpret_cast<const uint32_t*>(&b);
}

// `nrows` rows of D values, contiguous at src, to rows `stride` elements
// apart at dst; threads tid, tid + n, ...
__device__ __forceinline__ void read_token_major(const void* src, bool fp8, float s, int nrows,
                                                 int D, uint16_t* dst, long long stride, int tid,
                                                 int n) {
  const int cpr = D / 16, total = nrows * cpr;  // 16 values a chunk
  for (int c = tid; c < total; c += n) {
    uint4 lo, hi;
    if (fp8) {
      const uint4 x = reinterpret_cast<const uint4*>(src)[c];
      lo = make_uint4(dequant2(x.x, s), dequant2(x.x >> 16, s), dequant2(x.y, s),
                      dequant2(x.y >> 16, s));
      hi = make_uint4(dequant2(x.z, s), dequant2(x.z >> 16, s), dequant2(x.w, s),
                      dequant2(x.w >> 16, s));
    } else {
      lo = reinterpret_cast<const uint4*>(src)[2 * c];
      hi = reinterpret_cast<const uint4*>(src)[2 * c + 1];
    }
    uint4* o = reinterpret_cast<uint4*>(dst + (long long)(c / cpr) * stride + 16 * (c % cpr));
    o[0] = lo;
    o[1] = hi;
  }
}

// A dim-major tile of 16 tokens x 128 dims (one warp): lane l holds dims
// 4l .. 4l+3 of every token and stores 8 bytes of each token's row.
__device__ __forceinline__ void read_v_16x128(const uint8_t* src, bool fp8, float s, int slot0,
                                              int nrows, uint16_t* dst, long long stride) {
  const int lane = threadIdx.x & 31;
  uint16_t* o = dst + 4 * lane;
  if (fp8) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = reinterpret_cast<const uint4*>(src)[4 * lane + k];
    const uint32_t(*w)[4] = reinterpret_cast<const uint32_t(*)[4]>(x);
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      if (t < slot0 || t >= slot0 + nrows) continue;
      const int sel = 0x0040 + (t & 3) * 0x0011;  // byte t & 3 of both words
      const uint32_t a = __byte_perm(w[0][t >> 2], w[1][t >> 2], sel);
      const uint32_t b = __byte_perm(w[2][t >> 2], w[3][t >> 2], sel);
      *reinterpret_cast<uint2*>(o + (t - slot0) * stride) =
          make_uint2(dequant2(a, s), dequant2(b, s));
    }
  } else {
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = reinterpret_cast<const uint4*>(src)[8 * lane + k];
    const uint32_t(*w)[8] = reinterpret_cast<const uint32_t(*)[8]>(x);
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      if (t < slot0 || t >= slot0 + nrows) continue;
      const int sel = (t & 1) ? 0x7632 : 0x5410;
      *reinterpret_cast<uint2*>(o + (t - slot0) * stride) =
          make_uint2(__byte_perm(w[0][t >> 1], w[1][t >> 1], sel),
                     __byte_perm(w[2][t >> 1], w[3][t >> 1], sel));
    }
  }
}

// Any other dim-major tile, element by element (stores coalesced).
__device__ __noinline__ void read_v_any(const void* src, bool fp8, float s, int slot0, int nrows,
                                        int D, int P, uint16_t* dst, long long stride) {
  for (int e = threadIdx.x & 31; e < nrows * (D / 2); e += 32) {
    const int i = e / (D / 2), dd = 2 * (e % (D / 2)), at = dd * P + slot0 + i;
    uint32_t w;
    if (fp8) {
      const uint8_t* c = static_cast<const uint8_t*>(src);
      w = dequant2((uint32_t)c[at] | ((uint32_t)c[at + P] << 8), s);
    } else {
      const uint16_t* c = static_cast<const uint16_t*>(src);
      w = (uint32_t)c[at] | ((uint32_t)c[at + P] << 16);
    }
    *reinterpret_cast<uint32_t*>(dst + i * stride + dd) = w;
  }
}

__global__ void __launch_bounds__(kThreads) read_rows_kernel(const ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const kv_pool_desc& d = a.d;
  const int P = d.page_size;
  const int r = ragged_owner(a.out_indptr, a.B, P, blockIdx.x);
  const long long o0 = a.out_indptr[r], o1 = a.out_indptr[r + 1];
  const int local = blockIdx.x - ragged_first(o0, P, r);  // the request's touched page number
  if (a.abort_mask != nullptr && a.abort_mask[r] != 0) return;
  const long long start = a.row_start != nullptr ? a.row_start[r] : 0, n = o1 - o0;
  const long long L = a.seq_lens[r];
  if (n == 0) return;
  if (o0 < 0 || n < 0 || o1 > a.total_rows || start < 0 || start + n > L ||
      start + n > (long long)a.max_pages * P) {
    if (threadIdx.x == 0 && local == 0) set_error(d.ctl, KV_ERR_INVALID_ARG);
    return;
  }
  const long long j = start / P + local;
  const long long lo = max(j * P, start), hi = min((j + 1) * P, start + n);
  if (local < 0 || lo >= hi) return;
  const int p = a.page_table[(long long)r * a.max_pages + j];
  if (p < 0 || p >= d.num_pages) {
    if (threadIdx.x == 0) set_error(d.ctl, KV_ERR_BAD_PAGE_ID);
    return;
  }
  const bool fp8 = d.dtype == KV_DTYPE_E4M3;
  const int es = fp8 ? 1 : 2, Dk = d.head_dim_k, Dv = d.head_dim_v, H = d.num_kv_heads;
  const int nrows = (int)(hi - lo), slot0 = (int)(lo - j * P);
  const long long row = o0 + (lo - start);
  const uint8_t* kc = static_cast<const uint8_t*>(d.k_cache);
  if (d.layout == KV_LAYOUT_LATENT) {
    read_token_major(kc + ((long long)p * P + slot0) * Dk * es, fp8, fp8 ? d.k_scale[p] : 1.0f,
                     nrows, Dk, a.k_out + row * Dk, Dk, threadIdx.x, kThreads);
    return;
  }
  const uint8_t* vc = static_cast<const uint8_t*>(d.v_cache);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = warp; t < 2 * H; t += kThreads / 32) {
    const int h = t >> 1;
    const long long ph = (long long)p * H + h;
    if ((t & 1) == 0) {
      read_token_major(kc + (ph * P + slot0) * Dk * es, fp8, fp8 ? d.k_scale[ph] : 1.0f, nrows,
                       Dk, a.k_out + (row * H + h) * Dk, (long long)H * Dk, lane, 32);
    } else {
      const uint8_t* src = vc + ph * P * Dv * es;
      const float s = fp8 ? d.v_scale[ph] : 1.0f;
      uint16_t* dst = a.v_out + (row * H + h) * Dv;
      if (P == 16 && Dv == 128)
        read_v_16x128(src, fp8, s, slot0, nrows, dst, (long long)H * Dv);
      else
        read_v_any(src, fp8, s, slot0, nrows, Dv, P, dst, (long long)H * Dv);
    }
  }
}

}  // namespace

cudaError_t launch_read_rows(const ReadArgs& a, cudaStream_t s, int* launches) {
  const unsigned items = (unsigned)ragged_items(a.total_rows, a.B, a.d.page_size);
  const cudaError_t e = launch_pdl(read_rows_kernel, dim3(items), dim3(kThreads), 0, s, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
