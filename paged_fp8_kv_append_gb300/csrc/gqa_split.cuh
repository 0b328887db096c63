// gqa_split.cuh -- what the split kernels over grouped heads share (e4m3 and
// bf16 pools: decode_gqa.cu; 4-bit pools: decode_e2m1.cu): the walk over a
// batch's segments, conversions and products, and the end of a piece.
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

// ------------------------------------------------- tensor-core helpers


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

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ uint4 lds128(const void* p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p)));
  return v;
}
__device__ __forceinline__ uint2 lds64(const void* p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(p)));
  return v;
}
__device__ __forceinline__ uint32_t lds32(const void* p) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)));
  return v;
}

__device__ __forceinline__ uint32_t w_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// End of a piece: merges the online-softmax states of the WPH warps that
// share each of the Hv virtual heads (8 rows each) into the piece's partial.
// merge_ml[(w * 8 + nw) * 2 + {0, 1}] holds warp w's running max and sum of
// row nw, merge_o[(w * 8 + nw) * 128 + dd] its unnormalised output.  Pass 1,
// one thread per row: the row's max M over the warps, each warp's weight
// 2^(m_w - M) (written over m_w) and the weighted sum, stored with M (a
// piece that met a page it must not read stores the sum -1 instead).  Pass
// 2, every consumer thread: the weighted outputs, four dims at a time.
// row_of(v, nw) is the partial row of virtual head v's row nw.  Starts and
// ends with the consumer warps synchronised.
template <class C, class RowOf>
__device__ __forceinline__ void merge_piece(float* merge_o, float* merge_ml, int Hv, int WPH,
                                            const DecodeArgs& a, RowOf row_of,
                                            volatile int* piece_bad, bool reset_bad) {
  constexpr int R8 = C::R8, D = C::D, NT = C::CONSUMERS * 32;
  static_assert(R8 == 8 && D == 128, "index shifts");
  const int tid = threadIdx.x;
  named_bar_sync(1, NT);  // every warp's state is in the merge buffers
  if (tid < Hv * R8) {
    const int v = tid >> 3, nw = tid & 7;
    float M = -INFINITY;
    for (int q = 0; q < WPH; ++q) M = fmaxf(M, merge_ml[((q * Hv + v) * R8 + nw) * 2]);
    float lsum = 0.0f;
    for (int q = 0; q < WPH; ++q) {
      float* ml = merge_ml + ((q * Hv + v) * R8 + nw) * 2;
      const float w = (ml[0] == -INFINITY) ? 0.0f : exp2f(ml[0] - M);
      lsum += ml[1] * w;
      ml[0] = w;
    }
    const long long row = row_of(v, nw);
    a.ws.ml_part[row * 2 + 0] = M;
    a.ws.ml_part[row * 2 + 1] = *piece_bad ? -1.0f : lsum;
  }
  named_bar_sync(1, NT);
  if (reset_bad && tid == 0) *piece_bad = 0;
  for (int e = tid; e < Hv * R8 * (D / 4); e += NT) {
    const int d4 = e & 31, rr = e >> 5, v = rr >> 3, nw = rr & 7;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int q = 0; q < WPH; ++q) {
      const int w = (q * Hv + v) * R8 + nw;
      const float wt = merge_ml[w * 2];
      const float4 x = *reinterpret_cast<const float4*>(merge_o + w * D + 4 * d4);
      o.x = fmaf(wt, x.x, o.x);
      o.y = fmaf(wt, x.y, o.y);
      o.z = fmaf(wt, x.z, o.z);
      o.w = fmaf(wt, x.w, o.w);
    }
    *reinterpret_cast<float4*>(a.ws.o_part + row_of(v, nw) * D + 4 * d4) = o;
  }
  named_bar_sync(1, NT);
}

}  // namespace
}  // namespace kvfp8
