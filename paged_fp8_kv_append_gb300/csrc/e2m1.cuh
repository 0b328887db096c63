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

// 1 / s, correctly rounded, for s = 1/512 .. 448 of e4m3: the hardware's
// approximation and one step of Newton's iteration with an exact remainder.
// (Compared with the division for every e4m3 value in the tests.)
__device__ __forceinline__ float reciprocal_e4m3(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.0f), r, r);
}

// Two groups' scale bytes (the first in the low byte) and factors f from their
// largest magnitudes; c = 1 / (6 S), rounded once.  A group with a value that is
// not finite gets a scale of NaN (its codes then mean nothing).
__device__ __forceinline__ uint32_t e2m1_group_scales(float m0, float m1, float c, float inv_s,
                                                      float& f0, float& f1) {
  const bool ok0 = m0 <= 3.402823466e38f, ok1 = m1 <= 3.402823466e38f;
  uint32_t code = e4m3x2(m0 * c, m1 * c);  // saturating
  const float2 s = __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)code, __NV_E4M3)));
  f0 = ok0 && s.x > 0.0f ? reciprocal_e4m3(s.x) * inv_s : 0.0f;
  f1 = ok1 && s.y > 0.0f ? reciprocal_e4m3(s.y) * inv_s : 0.0f;
  if (!ok0) code = (code & 0xFF00u) | 0x7Fu;
  if (!ok1) code = (code & 0x00FFu) | 0x7F00u;
  return code;
}
constexpr float kE2m1Sixth = 1.0f / 6.0f;

// Two products (the packed multiplier; each rounded once)
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// the two bf16 values of w
__device__ __forceinline__ uint64_t bf16x2_values(uint32_t w) { return pack2(bf16_lo(w), bf16_hi(w)); }

// Eight codes of four pairs, the first value of a pair in the low half of its byte.
__device__ __forceinline__ uint32_t e2m1x8(uint64_t a, uint64_t b, uint64_t c, uint64_t d) {
  uint32_t r;
  asm("{\n .reg .b8 x, y, z, t;\n .reg .f32 lo, hi;\n"
      " mov.b64 {lo, hi}, %1;\n cvt.rn.satfinite.e2m1x2.f32 x, hi, lo;\n"
      " mov.b64 {lo, hi}, %2;\n cvt.rn.satfinite.e2m1x2.f32 y, hi, lo;\n"
      " mov.b64 {lo, hi}, %3;\n cvt.rn.satfinite.e2m1x2.f32 z, hi, lo;\n"
      " mov.b64 {lo, hi}, %4;\n cvt.rn.satfinite.e2m1x2.f32 t, hi, lo;\n"
      " mov.b32 %0, {x, y, z, t};\n}\n"
      : "=r"(r)
      : "l"(a), "l"(b), "l"(c), "l"(d));
  return r;
}

// The larger magnitudes of two bf16 pairs (with a sign of no meaning); NaN if one is.
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t larger8(const uint4& v) {
  return larger2(larger2(v.x, v.y), larger2(v.z, v.w));
}
__device__ __forceinline__ float low_magnitude(uint32_t w) { return __uint_as_float((w & 0x7FFFu) << 16); }
__device__ __forceinline__ float high_magnitude(uint32_t w) { return __uint_as_float(w & 0x7FFF0000u); }
// Largest magnitude of 16 bf16 values; NaN if one is.
__device__ __forceinline__ float amax16_bf16(const uint4& a, const uint4& b) {
  const uint32_t m = larger2(larger8(a), larger8(b));
  return low_magnitude(larger2(m, m >> 16));
}
__device__ __forceinline__ float finite_or_zero(float m) { return m <= 3.402823466e38f ? m : 0.0f; }

// 8 bf16 values times f as 8 codes, value k at nibble k
__device__ __forceinline__ uint32_t e2m1_codes8(const uint4& v, float f) {
  const uint64_t ff = pack2(f, f);
  return e2m1x8(mul2(bf16x2_values(v.x), ff), mul2(bf16x2_values(v.y), ff),
                mul2(bf16x2_values(v.z), ff), mul2(bf16x2_values(v.w), ff));
}

// The block scale that a tile's new rows go by: theirs in a fresh page (and
// stored), else the page's own.
__device__ __forceinline__ float e2m1_tile_scale(float amax, bool fresh, float* scale_slot) {
  if (!fresh) return *scale_slot;
  // (magnitudes order as their bits)
  const float s = e2m1_block_scale(
      __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))));
  if ((threadIdx.x & 31) == 0) *scale_slot = s;
  return s;
}

// Rows in global memory, src_stride elements apart: 16-byte chunk c of row i.
struct GlobalRows {
  const uint16_t* src;
  long long stride;
  __device__ __forceinline__ uint4 operator()(int i, int c) const {
    return reinterpret_cast<const uint4*>(src + i * stride)[c];
  }
};

// K rows slot0 .. slot0 + nrows - 1 of a tile; load(i, c): the 16-byte chunk c of row i.
// Lane (g, t): slots g and g + 8, groups t and t + 4: nothing is exchanged but
// the block's largest magnitude.  WHOLE: a fresh page's 16 rows.
template <bool WHOLE, class Load>
static __device__ __forceinline__ void e2m1_k_tile(const Load& load, int nrows, int slot0,
                                                   bool fresh, float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint4 v[2][2][2];  // [slot half][group half][16 bytes]
  bool mine[2];
  float m[2][2], block = 0.0f;
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int i = g + 8 * hi - slot0;
    mine[hi] = WHOLE || (i >= 0 && i < nrows);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        v[hi][c][u] = mine[hi] ? load(i, 2 * (t + 4 * c) + u) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int hi = 0; hi < 2; ++hi)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[hi][c] = amax16_bf16(v[hi][c][0], v[hi][c][1]);
      block = fmaxf(block, finite_or_zero(m[hi][c]));
    }
  const float inv_s = pow2_inverse(e2m1_tile_scale(block, WHOLE || fresh, scale_slot));
  const float sixth = inv_s * kE2m1Sixth;
  uint32_t sc[2];
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    float f0, f1;
    sc[hi] = e2m1_group_scales(m[hi][0], m[hi][1], sixth, inv_s, f0, f1);
    const uint4 code = make_uint4(e2m1_codes8(v[hi][0][0], f0), e2m1_codes8(v[hi][0][1], f0),
                                  e2m1_codes8(v[hi][1][0], f1), e2m1_codes8(v[hi][1][1], f1));
    if (mine[hi]) *reinterpret_cast<uint4*>(dst + 16 * lane + 512 * hi) = code;
    if (!WHOLE && mine[hi])
      *reinterpret_cast<uint16_t*>(dst + kE2m1Scales + 4 * lane + 2 * hi) = (uint16_t)sc[hi];
  }
  if (WHOLE) *reinterpret_cast<uint32_t*>(dst + kE2m1Scales + 4 * lane) = sc[0] | (sc[1] << 16);
}

// The V part of a tile from a lane's values: lane (c, t) holds the 16 dims of
// group c of its four slots 2t, 2t + 1, 2t + 8, 2t + 9 (tokens i = 0 .. 3):
// pair(h, k) are dim 16 c + k of tokens 2h and 2h + 1 in fp32, m[i] a slot's
// largest magnitude.  A byte holds two slots of a dim, so slots that are not
// written keep their halves (read back first).
template <bool WHOLE, class Pair>
static __device__ __forceinline__ void e2m1_v_store(Pair pair, const float (&m)[4],
                                                    const bool (&mine)[4], float inv_s,
                                                    uint8_t* dst) {
  const int lane = threadIdx.x & 31;
  if (!WHOLE && !(mine[0] || mine[1] || mine[2] || mine[3])) return;
  const float sixth = inv_s * kE2m1Sixth;
  float f[4];
  uint32_t sc = e2m1_group_scales(m[0], m[1], sixth, inv_s, f[0], f[1]);
  sc |= e2m1_group_scales(m[2], m[3], sixth, inv_s, f[2], f[3]) << 16;
  const uint64_t f01 = pack2(f[0], f[1]), f23 = pack2(f[2], f[3]);
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)  // byte b: tokens 2 (b / 2) and + 1, dim 2 k + b % 2
    w[k] = e2m1x8(mul2(pair(0, 2 * k), f01), mul2(pair(0, 2 * k + 1), f01),
                  mul2(pair(1, 2 * k), f23), mul2(pair(1, 2 * k + 1), f23));
  uint4* lo = reinterpret_cast<uint4*>(dst + 16 * lane);
  uint4* hi = lo + 32;
  uint32_t* scales = reinterpret_cast<uint32_t*>(dst + kE2m1Scales + 4 * lane);
  if (!WHOLE) {
    uint32_t keep = 0, keep_sc = 0;  // nibbles / bytes that stay as they are
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!mine[i]) {
        keep |= (i & 1 ? 0xF0F0u : 0x0F0Fu) << (16 * (i >> 1));
        keep_sc |= 0xFFu << (8 * i);
      }
    if (keep != 0) {
      const uint4 a = *lo, b = *hi;
      const uint32_t old[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = (w[k] & ~keep) | (old[k] & keep);
      sc = (sc & ~keep_sc) | (*scales & keep_sc);
    }
  }
  *lo = make_uint4(w[0], w[1], w[2], w[3]);
  *hi = make_uint4(w[4], w[5], w[6], w[7]);
  *scales = sc;
}

// V rows slot0 .. slot0 + nrows - 1 of a tile; load as for K.
template <bool WHOLE, class Load>
static __device__ __forceinline__ void e2m1_v_tile(const Load& load, int nrows, int slot0,
                                                   bool fresh, float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, c = lane >> 2, t = lane & 3;
  uint4 v[4][2];
  bool mine[4];
  float m[4], block = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 2 * t + (i & 1) + 8 * (i >> 1) - slot0;
    mine[i] = WHOLE || (row >= 0 && row < nrows);
#pragma unroll
    for (int u = 0; u < 2; ++u) v[i][u] = mine[i] ? load(row, 2 * c + u) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = amax16_bf16(v[i][0], v[i][1]);
    block = fmaxf(block, finite_or_zero(m[i]));
  }
  const float inv_s = pow2_inverse(e2m1_tile_scale(block, WHOLE || fresh, scale_slot));
  e2m1_v_store<WHOLE>(
      [&](int h, int k) {
        auto word = [&](const uint4& q) {
          const int j = (k & 7) >> 1;
          return j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
        };
        const uint32_t a = word(v[2 * h][k >> 3]), b = word(v[2 * h + 1][k >> 3]);
        return k & 1 ? pack2(bf16_hi(a), bf16_hi(b)) : pack2(bf16_lo(a), bf16_lo(b));
      },
      m, mine, inv_s, dst);
}

// The same for a fresh page from a bf16 pool's dim-major tile (16 slots of a dim
// together), of which the first nrows slots are rows; load(d, w): slots 2w and
// 2w + 1 of dim d.
template <bool WHOLE, class Load>
static __device__ __forceinline__ void e2m1_v_tile_dim_major(const Load& load, int nrows,
                                                             float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, c = lane >> 2, t = lane & 3;
  uint32_t v[2][16];  // [slot half][dim]: slots 2t, 2t + 1 of that half
  bool mine[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[i] = WHOLE || 2 * t + (i & 1) + 8 * (i >> 1) < nrows;
  uint32_t mm[2] = {0, 0};
#pragma unroll
  for (int hi = 0; hi < 2; ++hi)
#pragma unroll
    for (int k = 0; k < 16; ++k) v[hi][k] = load(16 * c + k, t + 4 * hi);
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    if (!WHOLE) {
      // (the whole tile is loaded: it lies in the page; slots that are no rows count as zeros)
      const uint32_t mask = (mine[2 * hi] ? 0xFFFFu : 0u) | (mine[2 * hi + 1] ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[hi][k] &= mask;
    }
    mm[hi] = larger2(v[hi][0], v[hi][1]);
#pragma unroll
    for (int k = 2; k < 16; ++k) mm[hi] = larger2(mm[hi], v[hi][k]);
  }
  const float m[4] = {low_magnitude(mm[0]), high_magnitude(mm[0]), low_magnitude(mm[1]),
                      high_magnitude(mm[1])};
  float block = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) block = fmaxf(block, finite_or_zero(m[i]));
  const float inv_s = pow2_inverse(e2m1_tile_scale(block, true, scale_slot));
  e2m1_v_store<WHOLE>([&](int h, int k) { return bf16x2_values(v[h][k]); }, m, mine, inv_s, dst);
}

}  // namespace kvfp8
