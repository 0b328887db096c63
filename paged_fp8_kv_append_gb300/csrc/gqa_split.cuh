// gqa_split.cuh -- what the split kernels over grouped heads share (e4m3 and
// bf16 pools: decode_gqa.cu; 4-bit pools: decode_e2m1.cu): the walk over a
// batch's segments, conversions, and the scaling of query rows.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace kvfp8 {
namespace {

// ------------------------------------------------- segment cursor

// Walks segments (request r, head group h) of the flattened unit sequence;
// `groups` is the number of head groups per request.  pfx may live in shared
// or global memory.
struct Cursor {
  int r, h, np;
  long long seg_start;
};

__device__ __forceinline__ Cursor cursor_at(const int32_t* pfx, int B, int groups, long long x) {
  // last r with pfx[r] <= x / groups; that request has pages (pfx[r+1] > x/groups)
  const long long v = x / groups;
  int lo = 0, hi = B;  // invariant: pfx[lo] <= v < pfx[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pfx[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  Cursor c;
  c.r = lo;
  c.np = pfx[lo + 1] - pfx[lo];
  c.h = (int)((x - (long long)groups * pfx[lo]) / c.np);
  c.seg_start = (long long)groups * pfx[lo] + (long long)c.h * c.np;
  return c;
}

__device__ __forceinline__ void cursor_next(Cursor& c, const int32_t* pfx, int B, int groups) {
  if (++c.h == groups) {
    c.h = 0;
    do {
      ++c.r;
    } while (c.r < B && pfx[c.r + 1] == pfx[c.r]);
    if (c.r < B) c.np = pfx[c.r + 1] - pfx[c.r];
  }
  if (c.r < B) {
    c.seg_start = (long long)groups * pfx[c.r] + (long long)c.h * c.np;
  } else {  // past the last request (cannot happen inside a CTA range): end every loop
    c.seg_start = (long long)groups * pfx[B];
    c.np = 1;
  }
}

// ------------------------------------------------- conversions

// Four e4m3 codes (bytes 0..3 of w) -> two f16x2 words, lo = (b0, b1) and
// hi = (b2, b3); exact (every e4m3 value is an f16 value).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 2^x on the special-function unit (flushes denormal results to zero, which
// only drops softmax weights below 2^-126).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The e4m3 paths multiply the bf16 query in f16.  Each query row is first
// scaled by an exact power of two 2^e that puts its largest magnitude in
// [2^15, 2^16): inside f16's range (below 65504) with all of its bits, and
// small elements stay clear of f16's subnormals.  The row's scores are then
// 2^e times the true ones and its score scale takes 2^-e.  For a row whose
// elements are all normal f16 values either way, scores are bit-identical to
// the unscaled ones (a power-of-two factor commutes with rounding).
// Largest magnitude of 8 bf16 values as a bit pattern with the sign cleared
// (bit-pattern order is magnitude order for finite values).
__device__ __forceinline__ uint32_t bf16_absbits_max8(const uint4& v) {
  const uint32_t a = max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu);
  const uint32_t b = max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu);
  const uint32_t c = max(v.z & 0x7FFFu, (v.z >> 16) & 0x7FFFu);
  const uint32_t d = max(v.w & 0x7FFFu, (v.w >> 16) & 0x7FFFu);
  return max(max(a, b), max(c, d));
}
// e for a row whose largest magnitude has bf16 bits mb: 15 - floor(log2),
// within [-112, 112] so that 2^e and 2^-e times the score scale stay normal
// fp32 numbers (all-zero or subnormal rows take 112).
__device__ __forceinline__ int q_row_exp(uint32_t mb) {
  const int E = (int)(mb >> 7);
  return E == 0 ? 112 : min(112, max(-112, 142 - E));
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ uint32_t bf16x2_to_f16x2_scaled(uint32_t w, float pw) {
  const float lo = __uint_as_float(w << 16) * pw, hi = __uint_as_float(w & 0xFFFF0000u) * pw;
  return f32x2_to_f16x2(lo, hi);
}

__device__ __forceinline__ uint32_t w_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

}  // namespace
}  // namespace kvfp8
