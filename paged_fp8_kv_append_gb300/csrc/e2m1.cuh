// e2m1.cuh -- the 4-bit tile of a KV_DTYPE_E2M1 pool: 16 tokens of 128 dims of
// one kv head, K or V, quantised by one warp from its source rows.
//
// A value is code * s * S: an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), the e4m3 scale s of its group (16 dims of one token) and the
// tile's block scale S, a power of two in fp32 that the first rows written
// into the page set: S = 2^(floor(log2 amax) - 6), so the largest group's
// scale amax_g / (6 S) lies in [10.6, 21.4), 21 times below e4m3's largest
// value for the rows that follow and 2^9 above its smallest normal one for
// the groups beside it.  A group's scale is of its own rows alone, so a
// token's 4-bit form does not change when others join its page.
// With q = x * f, f = fp32(1 / s) / S: a division by S is exact, so q is off
// from the quotient x / (s S) by at most two roundings, and code(q) from
// code(x / (s S)) only where that lies within them of a border of two codes.
//
// code * s has 2 + 4 significant bits: exact in f16, and in bf16 with S.
//
// Layout of the 1152 bytes (group c = d / 16): the bytes a lane (g, t) =
// (lane / 4, lane % 4) of a decode warp needs lie together, in the order of
// the matrix fragments.
//   K codes   64 slot + 16 (c % 4) + 8 (c / 4) + (d % 16) / 2, low half d even:
//             slots g and g + 8, groups t and t + 4: two 16-byte loads
//   K scales  1024 + 16 (slot % 8) + 4 (c % 4) + 2 (slot / 8) + c / 4:
//             4 bytes at 1024 + 4 lane
//   V codes   512 (d % 16 / 8) + 64 c + 16 (slot % 8 / 2) + 4 (d % 8 / 2)
//             + 2 (slot / 8) + d % 2, low half slot even:
//             group g, slots 2t, 2t + 1, 2t + 8, 2t + 9: two 16-byte loads
//   V scales  1024 + 16 c + 4 (slot % 8 / 2) + 2 (slot / 8) + slot % 2:
//             4 bytes at 1024 + 4 lane
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"
#include "quant.cuh"

namespace kvfp8 {

constexpr int kE2m1Tile = 1152;     // bytes of a tile
constexpr int kE2m1Scales = 1024;   // offset of its group scales
constexpr int kE2m1MinExp = -100, kE2m1MaxExp = 121;  // of a block scale

// The block scale for rows of largest magnitude amax (finite; 1 when it is 0).
// Clamped so that 1 / S and fp32(1 / s) / S stay normal numbers: rows below
// 2^-94 lose bits.
__device__ __forceinline__ float e2m1_block_scale(float amax) {
  const int e = min(max((int)(__float_as_uint(amax) >> 23) - 133, kE2m1MinExp), kE2m1MaxExp);
  return amax > 0.0f ? __uint_as_float((uint32_t)(e + 127) << 23) : 1.0f;
}
// 1 / S of a power of two
__device__ __forceinline__ float pow2_inverse(float s) {
  return __uint_as_float(0x7F000000u - __float_as_uint(s));
}

// A group's scale byte and factor f for its largest magnitude; a group with a
// value that is not finite gets a scale of NaN (its codes then mean nothing).
__device__ __forceinline__ uint32_t e2m1_group_scale(float amax, float inv_s, float& f) {
  // e4m3 of the float2's low half; saturating
  const uint32_t c = e4m3x2(amax * inv_s * (1.0f / 6.0f), 0.0f) & 0xFFu;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
  const bool finite = amax <= 3.402823466e38f;
  f = finite && s > 0.0f ? __frcp_rn(s) * inv_s : 0.0f;
  return finite ? c : 0x7Fu;
}

// two codes: a in the low half
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  return __nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
}

// Largest magnitude of 16 bf16 values (bit patterns; above 0x7F80: a NaN).
__device__ __forceinline__ float amax16_bf16(const uint4& a, const uint4& b) {
  const uint32_t m = absbits_max8(absbits_max8(0u, a), b);
  return __uint_as_float(max(m & 0xFFFFu, m >> 16) << 16);
}
__device__ __forceinline__ float finite_or_zero(float m) { return m <= 3.402823466e38f ? m : 0.0f; }

// 8 bf16 values times f as 8 codes, value k at nibble k
__device__ __forceinline__ uint32_t e2m1_codes8(const uint4& v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = e2m1x2(bf16_lo(w[k]) * f, bf16_hi(w[k]) * f);
  return c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
}

// The block scale that a tile's new rows go by: theirs in a fresh page (and
// stored), else the page's own.
__device__ __forceinline__ float e2m1_tile_scale(float amax, bool fresh, float* scale_slot) {
  if (!fresh) return *scale_slot;
  const float s = e2m1_block_scale(warp_max(amax));
  if ((threadIdx.x & 31) == 0) *scale_slot = s;
  return s;
}

// K rows slot0 .. slot0 + nrows - 1 of a tile from bf16 rows src_stride apart.
// Lane (g, t): slots g and g + 8, groups t and t + 4: nothing is exchanged but
// the block's largest magnitude.
static __device__ __forceinline__ void e2m1_k_tile(const uint16_t* src, long long src_stride,
                                                   int nrows, int slot0, bool fresh,
                                                   float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint4 v[2][2][2];  // [slot half][group half][16 bytes]
  bool mine[2];
  float m[2][2], block = 0.0f;
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int i = g + 8 * hi - slot0;
    mine[hi] = i >= 0 && i < nrows;
    const uint4* row = reinterpret_cast<const uint4*>(src + (long long)(mine[hi] ? i : 0) * src_stride);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        v[hi][c][u] = mine[hi] ? row[2 * (t + 4 * c) + u] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int hi = 0; hi < 2; ++hi)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[hi][c] = amax16_bf16(v[hi][c][0], v[hi][c][1]);
      block = fmaxf(block, finite_or_zero(m[hi][c]));
    }
  const float inv_s = pow2_inverse(e2m1_tile_scale(block, fresh, scale_slot));
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    if (!mine[hi]) continue;
    uint32_t code[4], sc = 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float f;
      sc |= e2m1_group_scale(m[hi][c], inv_s, f) << (8 * c);
      code[2 * c] = e2m1_codes8(v[hi][c][0], f);
      code[2 * c + 1] = e2m1_codes8(v[hi][c][1], f);
    }
    *reinterpret_cast<uint4*>(dst + 64 * (g + 8 * hi) + 16 * t) =
        make_uint4(code[0], code[1], code[2], code[3]);
    *reinterpret_cast<uint16_t*>(dst + kE2m1Scales + 4 * lane + 2 * hi) = (uint16_t)sc;
  }
}

// The V part of a tile from a lane's values: lane (c, t) holds the 16 dims of
// group c of its four slots 2t, 2t + 1, 2t + 8, 2t + 9 (tokens i = 0 .. 3):
// value(i, k) is dim 16 c + k in fp32, m[i] a slot's largest magnitude.  A
// byte holds two slots of a dim, so slots that are not written keep their
// halves (read back first).
template <class Value>
static __device__ __forceinline__ void e2m1_v_store(Value value, const float (&m)[4],
                                                    const bool (&mine)[4], float inv_s,
                                                    uint8_t* dst) {
  const int lane = threadIdx.x & 31;
  if (!(mine[0] || mine[1] || mine[2] || mine[3])) return;
  float f[4];
  uint32_t sc = 0, keep = 0, keep_sc = 0;  // nibbles / bytes that stay as they are
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sc |= e2m1_group_scale(m[i], inv_s, f[i]) << (8 * i);
    if (!mine[i]) {
      keep |= (i & 1 ? 0xF0F0u : 0x0F0Fu) << (16 * (i >> 1));
      keep_sc |= 0xFFu << (8 * i);
    }
  }
  uint32_t* words = reinterpret_cast<uint32_t*>(dst + 16 * lane);  // words k: + 128 (k / 4) + k % 4
  uint32_t* scales = reinterpret_cast<uint32_t*>(dst + kE2m1Scales + 4 * lane);
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    w[k] = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // byte b: slots 2 (b / 2) and + 1, dim 2 k + b % 2
      const int i = 2 * (b >> 1), dd = 2 * k + (b & 1);
      w[k] |= e2m1x2(value(i, dd) * f[i], value(i + 1, dd) * f[i + 1]) << (8 * b);
    }
  }
  uint4* lo = reinterpret_cast<uint4*>(words);
  uint4* hi = reinterpret_cast<uint4*>(words + 128);
  if (keep != 0) {
    const uint4 a = *lo, b = *hi;
    const uint32_t old[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = (w[k] & ~keep) | (old[k] & keep);
    sc = (sc & ~keep_sc) | (*scales & keep_sc);
  }
  *lo = make_uint4(w[0], w[1], w[2], w[3]);
  *hi = make_uint4(w[4], w[5], w[6], w[7]);
  *scales = sc;
}

// V rows slot0 .. slot0 + nrows - 1 of a tile from bf16 rows src_stride apart.
static __device__ __forceinline__ void e2m1_v_tile(const uint16_t* src, long long src_stride,
                                                   int nrows, int slot0, bool fresh,
                                                   float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, c = lane >> 2, t = lane & 3;
  uint4 v[4][2];
  bool mine[4];
  float m[4], block = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 2 * t + (i & 1) + 8 * (i >> 1) - slot0;
    mine[i] = row >= 0 && row < nrows;
    const uint4* p = reinterpret_cast<const uint4*>(src + (long long)(mine[i] ? row : 0) * src_stride);
#pragma unroll
    for (int u = 0; u < 2; ++u) v[i][u] = mine[i] ? p[2 * c + u] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = amax16_bf16(v[i][0], v[i][1]);
    block = fmaxf(block, finite_or_zero(m[i]));
  }
  const float inv_s = pow2_inverse(e2m1_tile_scale(block, fresh, scale_slot));
  e2m1_v_store(
      [&](int i, int k) {
        const uint4& q = v[i][k >> 3];
        const int j = (k & 7) >> 1;
        const uint32_t w = j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
        return k & 1 ? bf16_hi(w) : bf16_lo(w);
      },
      m, mine, inv_s, dst);
}

// The same for a fresh page from a bf16 pool's dim-major tile (dim d's slots at
// src[16 d ..]), of which the first nrows slots are rows.
static __device__ __forceinline__ void e2m1_v_tile_dim_major(const uint16_t* src, int nrows,
                                                             float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, c = lane >> 2, t = lane & 3;
  const uint32_t* p = reinterpret_cast<const uint32_t*>(src + 256 * c) + t;
  uint32_t v[2][16];  // [slot half][dim]: slots 2t, 2t + 1 of that half
  bool mine[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[i] = 2 * t + (i & 1) + 8 * (i >> 1) < nrows;
  uint32_t mm[2] = {0, 0};
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    // (the whole tile is loaded: it lies in the page; slots that are no rows count as zeros)
    const uint32_t mask = (mine[2 * hi] ? 0xFFFFu : 0u) | (mine[2 * hi + 1] ? 0xFFFF0000u : 0u);
#pragma unroll
    for (int k = 0; k < 16; ++k) v[hi][k] = p[8 * k + 4 * hi] & mask;
#pragma unroll
    for (int k = 0; k < 16; ++k) mm[hi] = absbits_max2(mm[hi], v[hi][k]);
  }
  float m[4], block = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = i & 1 ? mm[i >> 1] >> 16 : mm[i >> 1] & 0xFFFFu;
    m[i] = __uint_as_float(b << 16);
    block = fmaxf(block, finite_or_zero(m[i]));
  }
  const float inv_s = pow2_inverse(e2m1_tile_scale(block, true, scale_slot));
  e2m1_v_store(
      [&](int i, int k) {
        const uint32_t w = v[i >> 1][k];
        return i & 1 ? bf16_hi(w) : bf16_lo(w);
      },
      m, mine, inv_s, dst);
}

}  // namespace kvfp8
