// read.cu -- kv_read_rows: cached rows back as contiguous bf16 rows.
//
// "Smaller, faster, safer: running Kimi and GLM at scale", section
// "Quantizing the KV cache": prefill works on a bf16 cache and decode on an
// e4m3 one.  Rows that leave the pool (to a bf16 prefill that reuses a prefix,
// to another worker) are x = bf16(code * scale), one multiplication in fp32
// and one rounding; bf16 pools copy the bits.
//
// Bounded by HBM: per row width codes in, 2 * width bytes out.  One CTA per
// touched page: a page's tiles are contiguous, and a warp's loads and stores
// are runs of whole sectors (8 values a lane for token-major rows; a dim-major
// V tile is transposed in registers, a lane holding 4 dims of all 16 tokens).
// A tile's loads are issued together, K and V of a head by the same warp.  Tiles other than 16 x
// 128 store V element by element: 16 x 256 4.0 TB/s, 16 x 64 3.4, 64 x 128 1.5 (e4m3; 16 x 128
// 6.1-6.3, bf16 6.0, latent rows 6.3).
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
__device__ __forceinline__ uint4 dequant8(uint2 w, float s) {
  return make_uint4(dequant2(w.x, s), dequant2(w.x >> 16, s), dequant2(w.y, s),
                    dequant2(w.y >> 16, s));
}

// 8 cached values, and their bf16 values
template <bool FP8>
struct Chunk {
  uint2 lo, hi;  // (hi: bf16 only)
  __device__ __forceinline__ void load(const void* src, int c) {
    if (FP8) {
      lo = __ldcs(static_cast<const uint2*>(src) + c);
    } else {
      const uint4 x = __ldcs(static_cast<const uint4*>(src) + c);
      lo = make_uint2(x.x, x.y);
      hi = make_uint2(x.z, x.w);
    }
  }
  __device__ __forceinline__ uint4 value(float s) const {
    return FP8 ? dequant8(lo, s) : make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
};

// `nrows` rows of D values, contiguous at src, to rows `stride` elements
// apart at dst; threads tid, tid + n, .., kU chunks' loads in flight (kD: D
// when it is known)
template <bool FP8, int kD, int kU>
__device__ __forceinline__ void read_rows_of(const void* src, float s, int nrows, int D,
                                             uint16_t* dst, long long stride, int tid, int n) {
  const int cpr = (kD ? kD : D) / 8, total = nrows * cpr;
  for (int c0 = tid; c0 < total; c0 += kU * n) {
    Chunk<FP8> x[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (c0 + k * n < total) x[k].load(src, c0 + k * n);
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int c = c0 + k * n, r = c / cpr;
      if (c < total)
        __stcs(reinterpret_cast<uint4*>(dst + r * stride + 8 * (c - r * cpr)), x[k].value(s));
    }
  }
}

// A head's 16 x 128 tiles of K and V by one warp: tokens slot0 .. slot0 + nrows - 1 to rows
// `stride` elements apart.  (The whole tiles are loaded: they lie in the page.)
template <bool FP8>
__device__ __forceinline__ void read_head_16x128(const uint8_t* ksrc, const uint8_t* vsrc,
                                                 float ks, float vs, int slot0, int nrows,
                                                 uint16_t* kdst, uint16_t* vdst,
                                                 long long stride) {
  constexpr int kN = FP8 ? 4 : 8;  // 16-byte pieces of a lane's 4 dims
  const int lane = threadIdx.x & 31;
  Chunk<FP8> k[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) k[i].load(ksrc, lane + 32 * i);
  uint32_t w[kN][4];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(vsrc) + kN * lane + i);
    w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = 2 * i + (lane >> 4) - slot0;
    if (t >= 0 && t < nrows)
      __stcs(reinterpret_cast<uint4*>(kdst + t * stride + 8 * (lane & 15)), k[i].value(ks));
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int t = i - slot0;
    uint32_t a, b;  // dims 4 lane, +1 and +2, +3 of token i
    if (FP8) {
      const int sel = 0x0040 + (i & 3) * 0x0011;  // byte i & 3 of both words
      a = dequant2(__byte_perm(w[0][i >> 2], w[1][i >> 2], sel), vs);
      b = dequant2(__byte_perm(w[2][i >> 2], w[3][i >> 2], sel), vs);
    } else {
      // dim d of the lane: pieces 2 d (tokens 0-7) and 2 d + 1
      const int sel = (i & 1) ? 0x7632 : 0x5410, h = i >> 3, q = (i & 7) >> 1;
      a = __byte_perm(w[0 + h][q], w[(2 + h) % kN][q], sel);
      b = __byte_perm(w[(4 + h) % kN][q], w[(6 + h) % kN][q], sel);
    }
    if (t >= 0 && t < nrows)
      __stcs(reinterpret_cast<uint2*>(vdst + t * stride + 4 * lane), make_uint2(a, b));
  }
}

// Any other dim-major tile, element by element (stores coalesced).
template <bool FP8>
__device__ __forceinline__ void read_v_any(const void* src, float s, int slot0, int nrows, int D,
                                        int P, uint16_t* dst, long long stride) {
  for (int e = threadIdx.x & 31; e < nrows * (D / 2); e += 32) {
    const int i = e / (D / 2), dd = 2 * (e % (D / 2)), at = dd * P + slot0 + i;
    uint32_t w;
    if (FP8) {
      const uint8_t* c = static_cast<const uint8_t*>(src);
      w = dequant2((uint32_t)c[at] | ((uint32_t)c[at + P] << 8), s);
    } else {
      const uint16_t* c = static_cast<const uint16_t*>(src);
      w = (uint32_t)c[at] | ((uint32_t)c[at + P] << 16);
    }
    *reinterpret_cast<uint32_t*>(dst + i * stride + dd) = w;
  }
}

// A request's rows, and whether they can be read (one that is aborted or has none: n 0, fits).
struct Request {
  long long o0, n, start;
  bool in_order, fits;
};
__device__ __forceinline__ Request request(const ReadArgs& a, int r) {
  Request q;
  const long long o1 = a.out_indptr[r + 1], L = a.seq_lens[r];
  q.o0 = a.out_indptr[r];
  q.start = a.row_start != nullptr ? a.row_start[r] : 0;
  q.in_order = q.o0 <= o1;
  q.n = a.abort_mask != nullptr && a.abort_mask[r] != 0 ? 0 : o1 - q.o0;
  q.fits = q.n == 0 || (q.n > 0 && q.o0 >= 0 && o1 <= a.total_rows && q.start >= 0 &&
                        q.start + q.n <= L && q.start + q.n <= (long long)a.max_pages * a.d.page_size);
  return q;
}

enum Shape { kTile16x128, kLatent, kAny };

// Registers for the loads in flight matter more than warps: 3 (bf16: 2) CTAs an
// SM read the 16 x 128 tiles back at 6.3 TB/s, 4 (3) at 6.0, 2 at 6.1 (bytes
// read and written, 32 requests of 4k to 32k rows, 8 heads).
template <bool FP8, int SHAPE>
__global__ void __launch_bounds__(kThreads, SHAPE == kLatent ? 2 : FP8 ? 3 : 2)
    read_rows_kernel(const ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const kv_pool_desc& d = a.d;
  const int P = SHAPE == kTile16x128 ? 16 : d.page_size;
  // the last block (its item is seldom one) looks at every request: a refused one's rows may lie
  // behind every item, or in another's
  if (blockIdx.x == gridDim.x - 1)
    for (int r = threadIdx.x; r < a.B; r += kThreads) {
      const Request q = request(a, r);
      if (!q.in_order || !q.fits) set_error(d.ctl, KV_ERR_INVALID_ARG);
    }
  const int r = ragged_owner_in_order(a.out_indptr, a.B, P, blockIdx.x);
  if (r < 0) return;
  const Request q = request(a, r);
  const long long o0 = q.o0, n = q.n, start = q.start;
  if (!q.fits || n == 0) return;
  const int local = blockIdx.x - ragged_first(o0, P, r);  // the request's touched page number
  const long long j = start / P + local;
  const long long lo = max(j * P, start), hi = min((j + 1) * P, start + n);
  if (local < 0 || lo >= hi) return;
  const int p = a.page_table[(long long)r * a.max_pages + j];
  if (p < 0 || p >= d.num_pages) {
    if (threadIdx.x == 0) set_error(d.ctl, KV_ERR_BAD_PAGE_ID);
    return;
  }
  constexpr int es = FP8 ? 1 : 2;
  const int Dk = d.head_dim_k, Dv = d.head_dim_v, H = d.num_kv_heads;
  const int nrows = (int)(hi - lo), slot0 = (int)(lo - j * P);
  const long long row = o0 + (lo - start);
  const uint8_t* kc = static_cast<const uint8_t*>(d.k_cache);
  const uint8_t* vc = static_cast<const uint8_t*>(d.v_cache);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (SHAPE == kLatent) {
    const uint8_t* src = kc + ((long long)p * P + slot0) * Dk * es;
    const float s = FP8 ? d.k_scale[p] : 1.0f;
    uint16_t* dst = a.k_out + row * Dk;
    if (Dk == 576)
      read_rows_of<FP8, 576, 6>(src, s, nrows, Dk, dst, Dk, threadIdx.x, kThreads);
    else
      read_rows_of<FP8, 0, 2>(src, s, nrows, Dk, dst, Dk, threadIdx.x, kThreads);
  } else if (SHAPE == kTile16x128) {
    for (int h = warp; h < H; h += kThreads / 32) {
      const long long ph = (long long)p * H + h, at = (row * H + h) * 128;
      read_head_16x128<FP8>(kc + ph * 2048 * es, vc + ph * 2048 * es, FP8 ? d.k_scale[ph] : 1.0f,
                            FP8 ? d.v_scale[ph] : 1.0f, slot0, nrows, a.k_out + at, a.v_out + at,
                            H * 128ll);
    }
  } else {
    for (int t = warp; t < 2 * H; t += kThreads / 32) {
      const int h = t >> 1;
      const long long ph = (long long)p * H + h;
      if ((t & 1) == 0)
        read_rows_of<FP8, 0, 2>(kc + (ph * P + slot0) * Dk * es, FP8 ? d.k_scale[ph] : 1.0f, nrows,
                                Dk, a.k_out + (row * H + h) * Dk, (long long)H * Dk, lane, 32);
      else
        read_v_any<FP8>(vc + ph * P * Dv * es, FP8 ? d.v_scale[ph] : 1.0f, slot0, nrows, Dv, P,
                        a.v_out + (row * H + h) * Dv, (long long)H * Dv);
    }
  }
}

template <bool FP8>
cudaError_t launch(const ReadArgs& a, cudaStream_t s) {
  const kv_pool_desc& d = a.d;
  const dim3 grid((unsigned)ragged_items(a.total_rows, a.B, d.page_size)), block(kThreads);
  if (d.layout == KV_LAYOUT_LATENT)
    return launch_pdl(read_rows_kernel<FP8, kLatent>, grid, block, 0, s, a);
  if (d.page_size == 16 && d.head_dim_k == 128 && d.head_dim_v == 128)
    return launch_pdl(read_rows_kernel<FP8, kTile16x128>, grid, block, 0, s, a);
  return launch_pdl(read_rows_kernel<FP8, kAny>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_read_rows(const ReadArgs& a, cudaStream_t s, int* launches) {
  const cudaError_t e = a.d.dtype == KV_DTYPE_E4M3 ? launch<true>(a, s) : launch<false>(a, s);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
