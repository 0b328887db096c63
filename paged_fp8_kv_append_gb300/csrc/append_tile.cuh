// append_tile.cuh -- one (page, kv head, K|V) tile quantised by one warp from
// its bf16 source rows, and the re-encoding of a block whose scale grows.
// Shared by the append kernels (append.cu) and the rotary append (rotary.cu).
#pragma once

#include "common.cuh"
#include "quant.cuh"

namespace kvfp8 {

constexpr int kTileChunks = 8;   // 16-byte source chunks per lane (P * D <= 2048)

// KV_SCALE_REQUANTIZE: the code c of a block whose scale grows from s_old
// to s_new becomes e4m3(fp32(decode(c) * s_old) / s_new) (IEEE divide).
__device__ __forceinline__ uint8_t requant_code(uint8_t c, float s_old, float s_new) {
  const float v = __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))), s_old);
  return (uint8_t)(e4m3x2(__fdiv_rn(v, s_new), 0.0f) & 0xFFu);
}

// Re-encode the n_old slots already written in a block (token-major: rows of
// D codes; dim-major: D rows of P slots), threads tid, tid + nthreads, ...
static __device__ void requant_block(uint8_t* dst, int n_old, int D, bool dim_major, int P, float s_old,
                              float s_new, int tid, int nthreads) {
  for (int e = tid; e < n_old * D; e += nthreads) {
    const int o = dim_major ? (e / n_old) * P + e % n_old : e;
    dst[o] = requant_code(dst[o], s_old, s_new);
  }
}

// A whole 16 x 128 page whose scale is below 2^-90, element by element with
// the IEEE divide (kept out of line: it is rare and its code is long).
static __device__ __noinline__ void page_ieee(const uint16_t* src, long long src_stride, bool dim_major,
                                       float s, uint8_t* dst) {
  const int lane = threadIdx.x & 31;
  for (int e = lane; e < 16 * 128; e += 32) {
    const int i = e >> 7, dd = e & 127;
    const float x = bf16_bits_to_f32(src[i * src_stride + dd]);
    dst[dim_major ? dd * 16 + i : i * 128 + dd] =
        (uint8_t)(e4m3x2(__fdiv_rn(x, s), 0.0f) & 0xFFu);
  }
}

// A whole 16-token page of a 128-dim V tile, transposed in registers: lane l
// loads dims 4l..4l+3 of every row and writes those 4 dim rows of 16 slots.
static __device__ void v_page_16x128(const uint16_t* src, long long src_stride, bool fp8,
                              float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31;
  uint2 x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    x[i] = *reinterpret_cast<const uint2*>(src + i * src_stride + 4 * lane);
  if (!fp8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = k < 2 ? x[2 * j].x : x[2 * j].y, b = k < 2 ? x[2 * j + 1].x
                                                                      : x[2 * j + 1].y;
        w[j] = (k & 1) ? __byte_perm(a, b, 0x7632) : __byte_perm(a, b, 0x5410);
      }
      uint4* o = reinterpret_cast<uint4*>(dst + (4 * lane + k) * 32);
      o[0] = make_uint4(w[0], w[1], w[2], w[3]);
      o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return;
  }
  uint32_t mb = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) mb = absbits_max2(absbits_max2(mb, x[i].x), x[i].y);
  mb = absbits_warp_max(mb);
  float amax = __uint_as_float(mb << 16);
  if (mb > 0x7F80u) {  // a NaN: the float maximum skips it
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fmaxf(amax2(x[i].x), amax2(x[i].y)));
    amax = warp_max(m);
  }
  const float s = scale_from_amax(amax), rs = __frcp_rn(s);
  if (lane == 0) *scale_slot = s;
  if (!scale_fast_ok(s)) {
    page_ieee(src, src_stride, true, s, dst);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = k < 2 ? x[2 * j].x : x[2 * j].y, b = k < 2 ? x[2 * j + 1].x
                                                                    : x[2 * j + 1].y;
      c[j] = (k & 1) ? e4m3x2(div_fresh(bf16_hi(a), s, rs), div_fresh(bf16_hi(b), s, rs))
                     : e4m3x2(div_fresh(bf16_lo(a), s, rs), div_fresh(bf16_lo(b), s, rs));
    }
    *reinterpret_cast<uint4*>(dst + (4 * lane + k) * 16) =
        make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16),
                   c[6] | (c[7] << 16));
  }
}

// A whole 16-token page of a 128-dim K tile (token-major): lane l holds
// dims 8 (l % 16) .. +7 of rows l / 16, l / 16 + 2, ...
static __device__ void k_page_16x128(const uint16_t* src, long long src_stride, bool fp8,
                              float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, c = lane & 15, i0 = lane >> 4;
  uint4 x[8];
#pragma unroll
  for (int t = 0; t < 8; ++t)
    x[t] = *reinterpret_cast<const uint4*>(src + (2 * t + i0) * src_stride + 8 * c);
  if (!fp8) {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      *reinterpret_cast<uint4*>(dst + ((2 * t + i0) * 128 + 8 * c) * 2) = x[t];
    return;
  }
  uint32_t mb = 0;
#pragma unroll
  for (int t = 0; t < 8; ++t) mb = absbits_max8(mb, x[t]);
  mb = absbits_warp_max(mb);
  float amax = __uint_as_float(mb << 16);
  if (mb > 0x7F80u) {  // a NaN: the float maximum skips it
    float m = 0.0f;
#pragma unroll
    for (int t = 0; t < 8; ++t) m = fmaxf(m, amax8(x[t]));
    amax = warp_max(m);
  }
  const float s = scale_from_amax(amax), rs = __frcp_rn(s);
  if (lane == 0) *scale_slot = s;
  if (!scale_fast_ok(s)) {
    page_ieee(src, src_stride, false, s, dst);
    return;
  }
#pragma unroll
  for (int t = 0; t < 8; ++t)
    *reinterpret_cast<uint2*>(dst + (2 * t + i0) * 128 + 8 * c) =
        make_uint2(quant_word_fresh(x[t].x, s, rs) | (quant_word_fresh(x[t].y, s, rs) << 16),
                   quant_word_fresh(x[t].z, s, rs) | (quant_word_fresh(x[t].w, s, rs) << 16));
}

// Any other tile: part of a page, another page shape, or the re-quantising
// mode's re-encoding (kept out of line so the whole-page code stays small).
static __device__ __noinline__ void tile_warp_generic(const uint16_t* src, long long src_stride,
                                               int nrows, int D, bool fp8, bool fresh,
                                               float* scale_slot, uint8_t* dst, bool dim_major,
                                               int P, int slot0, uint8_t* wtile, bool requant) {
  const int lane = threadIdx.x & 31;
  const int cpr = D / 8, total = nrows * cpr;
  uint4 v[kTileChunks];
#pragma unroll
  for (int t = 0; t < kTileChunks; ++t) {
    const int q = lane + 32 * t;
    v[t] = q < total ? *reinterpret_cast<const uint4*>(src + (q / cpr) * src_stride + 8 * (q % cpr))
                     : make_uint4(0, 0, 0, 0);
  }
  float s = 1.0f;
  if (fp8) {
    if (fresh) {
      float m = 0.0f;
#pragma unroll
      for (int t = 0; t < kTileChunks; ++t) m = fmaxf(m, amax8(v[t]));
      s = scale_from_amax(warp_max(m));
      if (lane == 0) *scale_slot = s;
    } else {
      s = *scale_slot;
      if (requant) {  // a larger scale for the new rows: re-encode the old ones
        float m = 0.0f;
#pragma unroll
        for (int t = 0; t < kTileChunks; ++t) m = fmaxf(m, amax8(v[t]));
        const float s_new = scale_from_amax(warp_max(m));
        if (s_new > s) {
          requant_block(dst, slot0, D, dim_major, P, s, s_new, lane, 32);
          __syncwarp();
          if (lane == 0) *scale_slot = s_new;
          s = s_new;
        }
      }
    }
  }
  const float rs = __frcp_rn(s);
  if (!dim_major) {
#pragma unroll
    for (int t = 0; t < kTileChunks; ++t) {
      const int q = lane + 32 * t;
      if (q < total) {
        const long long o = (long long)(slot0 + q / cpr) * D + 8 * (q % cpr);
        if (fp8)
          *reinterpret_cast<uint2*>(dst + o) = quant8_rs(v[t], s, rs);
        else
          *reinterpret_cast<uint4*>(dst + 2 * o) = v[t];
      }
    }
    return;
  }
  // dim-major destination: element (row i, dim dd) at (dd * P + slot0 + i),
  // assembled in this warp's shared tile, or without one (wtile null)
  // stored element by element
  if (wtile == nullptr) {
#pragma unroll
    for (int t = 0; t < kTileChunks; ++t) {
      const int q = lane + 32 * t;
      if (q < total) {
        const int o = 8 * (q % cpr) * P + slot0 + q / cpr;
        if (fp8) {
          const uint2 c8 = quant8_rs(v[t], s, rs);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[o + k * P] = (uint8_t)(((k < 4 ? c8.x : c8.y) >> (8 * (k & 3))) & 0xFFu);
        } else {
          const uint32_t w[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
          uint16_t* d16 = reinterpret_cast<uint16_t*>(dst);
#pragma unroll
          for (int k = 0; k < 8; ++k) d16[o + k * P] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
      }
    }
    return;
  }
#pragma unroll
  for (int t = 0; t < kTileChunks; ++t) {
    const int q = lane + 32 * t;
    if (q < total) {
      const int i = q / cpr, c = q % cpr;
      const int o = 8 * c * P + slot0 + i;
      if (fp8) {
        const uint2 c8 = quant8_rs(v[t], s, rs);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          wtile[o + k * P] = (uint8_t)(((k < 4 ? c8.x : c8.y) >> (8 * (k & 3))) & 0xFFu);
      } else {
        const uint32_t w[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
        uint16_t* t16 = reinterpret_cast<uint16_t*>(wtile);
#pragma unroll
        for (int k = 0; k < 8; ++k) t16[o + k * P] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
  __syncwarp();
  const int es = fp8 ? 1 : 2;
  if (nrows == P && (D * P * es) % 16 == 0) {
    for (int k = lane; k < D * P * es / 16; k += 32)
      reinterpret_cast<uint4*>(dst)[k] = reinterpret_cast<const uint4*>(wtile)[k];
  } else {
    for (int e = lane; e < D * nrows; e += 32) {
      const int o = (e / nrows) * P + slot0 + e % nrows;
      if (fp8)
        dst[o] = wtile[o];
      else
        reinterpret_cast<uint16_t*>(dst)[o] = reinterpret_cast<const uint16_t*>(wtile)[o];
    }
  }
  __syncwarp();
}

}  // namespace kvfp8
