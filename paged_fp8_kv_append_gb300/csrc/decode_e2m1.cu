// decode_e2m1.cu -- split-K paged decode attention over a 4-bit pool
// (KV_DTYPE_E2M1): its split kernels and its combine; the batch plan is that of
// the other formats (decode_plan.cuh).
//
// "Smaller, faster, safer: running Kimi and GLM at scale", section "Quantizing
// the KV cache": the kernel converts values as it reads them.
//
// A 4-bit page takes 9/16 of the bytes of an e4m3 one and the same arithmetic, so at
// HBM speed a page of a kv head leaves 420 cycles of a scheduler, where the e4m3
// kernels' page leaves 750.
//
// Work: units of two pages of one request for a group of Hs kv heads, cut into equal
// ranges, one per persistent CTA; a warp serves one (kv head, block of query rows) of
// every few units.  There is no producer warp, and nothing is shared between warps
// but the batch plan: each copies its own head's tiles into a ring of its own (16
// bytes a lane, cp.async), keeps its own online softmax and writes its own partial,
// which the combine merges with the others of the segment.  (With a producer's bulk
// copies and partials merged in the CTA: 166 us for the batch below; with bulk copies
// of each warp's own, 1152 bytes: 134.)
//
// Two pages are taken together: their products are independent chains, and waits,
// bookkeeping and the softmax's vote are one for 32 tokens.
//
// A row's running reference is moved only when a score exceeds it by more than
// 2^kSlack, so most pages need one vote where a maximum over the lanes takes six
// shuffles.
//
// Codes become f16 by cvt.rn.f16x2.e2m1x2 (a byte each, as cheap as a move beside
// the products); K's and V's group scales multiply them there (exact: six
// significant bits).  K's block scales go to the scores.  V's say nothing about a
// token's weight, so they stay out of the weights and their reference: a warp's
// outputs are in units of a power of two near its pages' V block scales, what a page
// differs by goes into its group scales (exact too, 2^14 below to 2^4 above), and where
// it differs by more the outputs move to another unit first, pages one at a time.  (With the
// block scale as an exponent bias of the weights the batch below took 0.7 us less, the
// ragged one 1.5, and a page of V 2^20 below another lost its weights' bits.)
//
// Up to 8 query rows a kv head bound by HBM: 32 requests of 4k-32k tokens, 64 and 8
// heads, 128 us in all, 5.7 TB/s of the 6.8 of a plain copy (the split's loop alone at
// the copy's rate; its first loads, a chain of three misses, take 6 us, the combine
// 5).  16 warps of 128 registers: with 12 of 168 it is 151 us.  Above 8 rows bound by
// the warps' instructions: 12 query heads a kv head, 48 requests of up to 8k: 70 us, 3.4
// TB/s, the tensor pipe busy 37%, issue 46%; there 64 accumulators a lane want 168
// registers (16 warps of 128: 96 us, what spills finds no L1 beside the ring).
//
// Two blocks of 16 rows are served by one warp where that leaves at most two warps for a
// head's units (decode_config): each page is copied and its codes are converted once for
// 32 rows.  24 requests of 4 drafts, 32 rows: 88 us against 94; 64 rows: 147 against 169.
// With more warps a head it is no faster, and slower for short requests (8 of 2k-9k on one
// kv head: 32 us against 26; each of its warps begins and ends every piece).  An odd number
// of blocks would pad the last (48 rows 145 against 128).  The products' rate (37 us for the
// drafts) stays far: a product takes 8 cycles of a scheduler, and what is issued beside it
// about 0.65 of its own cycles more (2 products 16, 4 conversions with their
// multiplications 12.5, together 25).
#include <climits>

#include "common.cuh"
#include "decode_plan.cuh"
#include "e2m1.cuh"
#include "gqa_split.cuh"
#include "internal.h"

namespace kvfp8 {
namespace {

constexpr int kStage = 4 * kE2m1Tile;  // a unit: K of its two pages, then V
constexpr int kPfxCache = 1024;        // plan entries cached in shared memory

// What a warp knows of its units, 16 of one batch and 16 of the next: for each of a
// unit's two pages its tile (-1: none, or not to be read) and block scales.
struct UnitTable {
  float2 ks[32], vs[32];
  int2 tile[32];
};

// NB: blocks of 16 query rows a warp serves; 0: up to 8 rows.
template <int NB>
struct E2m1Cfg {
  static constexpr int ROWS = NB > 0 ? 16 * NB : 8;  // of a warp
  static constexpr int WARPS = NB == 0 ? 16 : NB == 1 ? 12 : 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ST = 2;  // units in a warp's ring (3 and 4 were no faster)
  static constexpr int QBYTES = 256 * ROWS;
  // shared memory carve-up (byte offsets)
  static constexpr int OFF_Q = WARPS * ST * kStage;          // [W] Q operands
  static constexpr int OFF_UNIT = OFF_Q + WARPS * QBYTES;    // [W] UnitTable
  static constexpr int OFF_PFX = OFF_UNIT + WARPS * (int)sizeof(UnitTable);
  static constexpr int OFF_WSUM = OFF_PFX + kPfxCache * 4;  // [32] plan scan warp sums
  static constexpr int SMEM = OFF_WSUM + 32 * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// the reference of a row that has seen no position: fp32's lowest, so that any finite score passes it
constexpr float kUnset = -3.402823466e38f;
// A reference is set 2^kBelow below the row's largest weight, and moved when a weight exceeds it
// by more than 2^kSlack: f16 then keeps its 11 bits for weights down to 2^-20 of the largest
// (2^-14 without the distance), and none passes its 65504.
constexpr float kBelow = 6.0f, kSlack = 15.0f;
// The unit of a warp's outputs, as a float's exponent field.  A page's group scales take the
// difference from kUnder below it to kOver above: 448 * 6 * 2^4 is below f16's largest and
// 0.5 * 2^-9 * 2^-14 its smallest, so every value is exact.  A part begins with a unit for its
// first pages, and a page that does not fit moves it so that it lies 2 inside: pages within 2^16
// of each other move it no more, and are taken two at a time.  (32 requests of 4k-32k with a page
// in 8 2^12 below the others: 125 us, as without; moved by each of them in turn, 180.)  The unit
// does not follow a page more than kFar below the largest page's: outputs in a unit (at most 2^31
// weights of 2^15 times values of 2^15.4) then stay below fp32's largest, and what such a page
// loses is below 2^-56 of the largest values.
constexpr int kUnder = 14, kOver = 4, kFar = 64;

struct FalseType {
  static constexpr bool value = false;
};
struct TrueType {
  static constexpr bool value = true;
};

// A row's reference at the end of a warp's part, with its sum: -inf where the part holds no
// position for the merge.  Scores that are NaN pass no vote and leave the reference unset, but
// not the sum, which has to reach the merge.
__device__ __forceinline__ float final_reference(float m, float sum) {
  return m != kUnset ? m : sum != sum ? 0.0f : -INFINITY;
}
// A row's score scale, with the 2^-e of its queries; mb: their largest magnitude's bits.  A query
// that is not finite makes NaN of every score (an infinite one could otherwise pass for a mask).
__device__ __forceinline__ float row_score_scale(float scale, int e, uint32_t mb) {
  return mb >= 0x7F80u ? __int_as_float(0x7FFFFFFF) : scale * pow2f(-e);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
// Eight e2m1 codes -> four f16x2 words, one a byte (low half: low nibble).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c,
                                              uint32_t& d) {
  asm("{\n .reg .b8 x, y, z, t;\n mov.b32 {x, y, z, t}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, x;\n cvt.rn.f16x2.e2m1x2 %1, y;\n"
      " cvt.rn.f16x2.e2m1x2 %2, z;\n cvt.rn.f16x2.e2m1x2 %3, t;\n}\n"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}
// The same, bytes 0 and 1 times slo, 2 and 3 times shi (exact: an e2m1 code
// times an e4m3 scale has six significant bits).
__device__ __forceinline__ void e2m1x8_scaled(uint32_t w, uint32_t slo, uint32_t shi, uint32_t& a,
                                              uint32_t& b, uint32_t& c, uint32_t& d) {
  e2m1x8_to_f16(w, a, b, c, d);
  a = mul_f16x2(a, slo);
  b = mul_f16x2(b, slo);
  c = mul_f16x2(c, shi);
  d = mul_f16x2(d, shi);
}
__device__ __forceinline__ int exponent_field(float s) {  // of a positive value
  return (int)(__float_as_uint(s) >> 23);
}
// 2^x in both halves, x <= 15; FAR: 0 below f16's normal range
template <bool FAR>
__device__ __forceinline__ uint32_t pow2_f16x2(int x) {
  return FAR && x < -14 ? 0u : (uint32_t)(x + 15) * 0x04000400u;
}
// 2^x as a factor of sums, x <= 127; 0 below fp32's normal range
__device__ __forceinline__ float pow2_or_zero(int x) { return x < -126 ? 0.0f : pow2f(x); }
// A partial is 2^m (o, sum): with o in units of 2^x it is 2^(m + x) (o, 2^-x sum), which is how it
// is left for units up to 2^+-kPlain and references that take x exactly.  Beyond, the merge's
// factors would flush what is small, or the sum would lose x: there outputs are multiplied out, but
// for a shift that keeps them below 2^115 (unit and sum give their size; 0 but for values above
// 2^90, or a sum that is NaN).
constexpr int kPlain = 24;
constexpr float kPlainReference = 1048576.0f;
__device__ __forceinline__ int partial_shift(int x, float m, float sum) {
  if (abs(x) <= kPlain && (fabsf(m) < kPlainReference || m == -INFINITY)) return x;
  return min(126, max(0, x + exponent_field(fabsf(sum)) - 127 - 102));
}
// Whether a page of V block scale `page` lies where its group scales take the difference
// (exponent fields)
__device__ __forceinline__ bool unit_fits(int page, int unit) {
  return (uint32_t)(page - unit + kUnder) <= kUnder + kOver;
}
// The unit for a page that does not (`largest` so far)
__device__ __forceinline__ int unit_for(int page, int unit, int& largest) {
  largest = max(largest, page);
  return max(page > unit ? page - (kOver - 2) : page + (kUnder - 2), largest - kFar);
}
// the low or the high half of w in both halves
__device__ __forceinline__ uint32_t half_of(uint32_t w, int hi) {
  return __byte_perm(w, w, hi ? 0x3232 : 0x1010);
}
// Scale bytes of the tokens 2t, 2t + 1, 2t + 8, 2t + 9 that lie below nv (the
// bytes behind a request's length are stale and may be NaN).
__device__ __forceinline__ uint32_t e2m1_token_mask(int nv, int t) {
  const int a = min(max(nv - 2 * t, 0), 2), b = min(max(nv - 8 - 2 * t, 0), 2);
  return ((1u << (8 * a)) - 1u) | (((1u << (8 * b)) - 1u) << 16);
}
// The first slot whose scale byte (of the lane's group, tokens as above) is NaN, over the group's
// four lanes; 16: none.  NaN bytes become 0.
__device__ __forceinline__ int e2m1_first_nan(uint32_t& scales, int t) {
  int first = 16;
#pragma unroll
  for (int k = 3; k >= 0; --k)
    if ((scales >> (8 * k) & 0x7Fu) == 0x7Fu) {
      first = min(first, 2 * t + (k & 1) + 8 * (k >> 1));
      scales &= ~(0xFFu << (8 * k));
    }
  first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
  return min(first, __shfl_xor_sync(0xffffffffu, first, 2));
}
// The 8 x 8 f16 matrix that the warp holds two to a lane (lane 4 r + c: row r,
// columns 2c and 2c + 1), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// c += a b (m16n8k16, f16 operands)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int OFFSET>
__device__ __forceinline__ uint4 lds128_at(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4+%5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at), "n"(OFFSET));
  return v;
}
template <int OFFSET>
__device__ __forceinline__ uint32_t lds32_at(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(at), "n"(OFFSET));
  return v;
}

__device__ __forceinline__ void copy16(uint32_t dst_smem, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst_smem),
               "l"(src), "l"(policy)
               : "memory");
}

// A page as a warp meets it: its head's tiles, and what is known of them.
// (shared-memory addresses are 32-bit, with the lane's offset in them: 16 bytes of
// codes a lane at k16 and k16 + 512, 4 of scales at k4, and V's behind K's of the unit)
struct E2m1Page {
  uint32_t k16, k4;
  float ks, vs;  // block scales
  int nv, pos0;  // tokens below the request's length, the first one's position
};

// Up to 8 query rows of a kv head: S^T = K Q^T (M = 16 tokens, N = 8 rows) and
// O^T += V^T P^T.  Lane (g, t): tokens g, g + 8 and rows 2t, 2t + 1 of the scores.
struct E2m1Rows8 {
  float &m0, &m1, &l0, &l1;
  float (&acc)[8][4];
  const uint32_t q16;      // Q as B operands, [k-steps 2w, 2w + 1][lane] 16-byte words (at this lane's)
  const float qsc0, qsc1;  // score scales of rows 2t, 2t + 1
  const int G, T, seen0;   // query token tq sees positions 0 .. seen0 + tq
  int unit = -1, largest = -1;  // of acc, and of the pages' V block scales (-1: no page yet)

  // EDGE: some position may lie behind the length or behind a row's last one
  template <int NP, bool EDGE>
  __device__ __forceinline__ void pages(const E2m1Page (&pg)[NP]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[NP][4];
    {
      uint4 kg[NP], kh[NP];
      uint32_t sg[NP], sh[NP];
      float sb[NP][4];
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        kg[u] = lds128_at<0>(pg[u].k16);
        kh[u] = lds128_at<512>(pg[u].k16);
        e4m3x4_to_f16(lds32_at<0>(pg[u].k4), sg[u], sh[u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][e] = sb[u][e] = 0.0f;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {  // a code word: k-steps 2w, 2w + 1
        const uint4 q = w == 0   ? lds128_at<0>(q16)
                        : w == 1 ? lds128_at<512>(q16)
                        : w == 2 ? lds128_at<1024>(q16)
                                 : lds128_at<1536>(q16);
#pragma unroll
        for (int u = 0; u < NP; ++u) {
          const uint32_t s0 = half_of(sg[u], w >> 1), s1 = half_of(sh[u], w >> 1);
          uint32_t x[4], y[4];
          e2m1x8_scaled(w_of(kg[u], w), s0, s0, x[0], x[1], x[2], x[3]);
          e2m1x8_scaled(w_of(kh[u], w), s1, s1, y[0], y[1], y[2], y[3]);
          mma_f16(s[u], x[0], y[0], x[1], y[1], q.x, q.y);
          mma_f16(sb[u], x[2], y[2], x[3], y[3], q.z, q.w);
        }
      }
#pragma unroll
      for (int u = 0; u < NP; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][e] += sb[u][e];
    }
    // ---- weights against the rows' references
    float p[NP][4], big = -INFINITY;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const float sc0 = pg[u].ks * qsc0, sc1 = pg[u].ks * qsc1;
#pragma unroll
      for (int e = 0; e < 4; ++e) p[u][e] = fmaf(s[u][e], e & 1 ? sc1 : sc0, e & 1 ? -m1 : -m0);
    }
    if constexpr (EDGE) {
      const int lim0 = seen0 + min(2 * t / G, T - 1), lim1 = seen0 + min((2 * t + 1) / G, T - 1);
#pragma unroll
      for (int u = 0; u < NP; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = g + 8 * (e >> 1);
          if (tok >= pg[u].nv || pg[u].pos0 + tok > (e & 1 ? lim1 : lim0)) p[u][e] = -INFINITY;
        }
    }
#pragma unroll
    for (int u = 0; u < NP; ++u)
      big = fmaxf(big, fmaxf(fmaxf(p[u][0], p[u][1]), fmaxf(p[u][2], p[u][3])));
    if (__any_sync(0xffffffffu, big > kSlack)) {
      float n0 = kUnset, n1 = kUnset;
#pragma unroll
      for (int u = 0; u < NP; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // the scores themselves
          const float y = s[u][e] * (pg[u].ks * (e & 1 ? qsc1 : qsc0));
          p[u][e] = p[u][e] == -INFINITY ? -INFINITY : y;
          if (e & 1) n1 = fmaxf(n1, p[u][e]);
          else n0 = fmaxf(n0, p[u][e]);
        }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
      }
      n0 = fmaxf(n0 - kBelow, m0);
      n1 = fmaxf(n1 - kBelow, m1);
      const float a0 = fast_exp2(m0 - n0), a1 = fast_exp2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= a0;
      l1 *= a1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i][0] *= a0;
        acc[i][1] *= a1;
        acc[i][2] *= a0;
        acc[i][3] *= a1;
      }
#pragma unroll
      for (int u = 0; u < NP; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[u][e] -= e & 1 ? n1 : n0;
    }
#pragma unroll
    for (int u = 0; u < NP; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[u][e] = fast_exp2(p[u][e]);
      l0 += p[u][0] + p[u][2];
      l1 += p[u][1] + p[u][3];
    }
    // ---- O^T += V^T P^T: row g's weights of tokens 2t, 2t + 1 and 2t + 8, 2t + 9
    if constexpr (EDGE) {  // (others fit: the caller looks)
      const int page = exponent_field(pg[0].vs);
      if (!unit_fits(page, unit)) {
        const int to = unit_for(page, unit, largest);
        const float f = pow2_or_zero(unit - to);
        unit = to;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] *= f;
      }
    }
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const uint32_t b0 = transpose8x8(f32x2_to_f16x2(p[u][0], p[u][1]));
      const uint32_t b1 = transpose8x8(f32x2_to_f16x2(p[u][2], p[u][3]));
      const uint4 v0 = lds128_at<2 * kE2m1Tile>(pg[u].k16);
      const uint4 v1 = lds128_at<2 * kE2m1Tile + 512>(pg[u].k16);
      const uint32_t sw = lds32_at<2 * kE2m1Tile>(pg[u].k4);
      auto add = [&](uint32_t scales, uint32_t c0, uint32_t c1) {
        uint32_t slo, shi;  // scales of group g's same tokens
        e4m3x4_to_f16(scales, slo, shi);
        const uint32_t f = pow2_f16x2<EDGE>(exponent_field(pg[u].vs) - unit);
        slo = mul_f16x2(slo, f);
        shi = mul_f16x2(shi, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // rows g, g + 8 of tile i: dims 16g + 2i, + 1
          uint32_t a0, a1, a2, a3;
          e2m1x8_scaled(w_of(i < 4 ? v0 : v1, i & 3), slo, shi, a0, a1, a2, a3);
          mma_f16(acc[i], a0, a1, a2, a3, c0, c1);
        }
      };
      if constexpr (!EDGE) {
        add(sw, b0, b1);
      } else {
        // A scale of NaN (a value that was not finite) times a weight of zero is NaN: it
        // is left out of the product, and reaches the rows that see its token.
        uint32_t clean = sw & e2m1_token_mask(pg[u].nv, t);
        const int first = e2m1_first_nan(clean, t);
        add(clean, b0, b1);
        if (__any_sync(0xffffffffu, first < 16)) {
          const bool x0 = first < 16 && pg[u].pos0 + first <= seen0 + min(2 * t / G, T - 1);
          const bool x1 = first < 16 && pg[u].pos0 + first <= seen0 + min((2 * t + 1) / G, T - 1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (x0) acc[i][0] = acc[i][2] = __int_as_float(0x7FFFFFFF);
            if (x1) acc[i][1] = acc[i][3] = __int_as_float(0x7FFFFFFF);
          }
        }
      }
    }
  }
  // the sums over the lanes, and the references as the merge wants them
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    m0 = final_reference(m0, l0);
    m1 = final_reference(m1, l1);
  }
};

// NB blocks of 16 query rows of a kv head, from row n0 on: S = Q K^T (M = 16 rows, N = 8 tokens)
// and O += P V (N = 8 dims, K = 16 tokens).  Lane (g, t): rows g, g + 8 of a block and tokens 2t,
// 2t + 1, 2t + 8, 2t + 9, so the weights are the second product's A operand as they are.  The
// operands made of a page's codes serve all blocks.
template <int NB>
struct E2m1Rows16 {
  float (&m)[NB][2], (&l)[NB][2];  // of rows g and g + 8 of each block
  float (&acc)[NB][16][4];
  const uint32_t q16;  // Q as A operands, [block][k-step][lane] 16-byte words (at this lane's)
  const float (&qsc)[NB][2];
  const int n0, G, T, seen0;
  int unit = -1, largest = -1;

  // the last position that row g + 8 hr of block b sees
  __device__ __forceinline__ int last(int b, int hr) const {
    return seen0 + min((n0 + 16 * b + (int)((threadIdx.x & 31) >> 2) + 8 * hr) / G, T - 1);
  }
  // EDGE: some position may lie behind the length or behind a row's last one
  template <int NP, bool EDGE>
  __device__ __forceinline__ void pages(const E2m1Page (&pg)[NP]) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    float s[NP][NB][2][4];
    {
      uint4 kg[NP], kh[NP];
      uint32_t sg[NP], sh[NP];
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        kg[u] = lds128_at<0>(pg[u].k16);
        kh[u] = lds128_at<512>(pg[u].k16);
        e4m3x4_to_f16(lds32_at<0>(pg[u].k4), sg[u], sh[u]);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][b][0][e] = s[u][b][1][e] = 0.0f;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {  // a code word: k-steps 2w, 2w + 1
        uint4 q0[NB], q1[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          q0[b] = lds128_at<0>(q16 + 4096 * b + 1024 * w);
          q1[b] = lds128_at<512>(q16 + 4096 * b + 1024 * w);
        }
#pragma unroll
        for (int u = 0; u < NP; ++u) {
          const uint32_t s0 = half_of(sg[u], w >> 1), s1 = half_of(sh[u], w >> 1);
          uint32_t x[4], y[4];
          e2m1x8_scaled(w_of(kg[u], w), s0, s0, x[0], x[1], x[2], x[3]);
          e2m1x8_scaled(w_of(kh[u], w), s1, s1, y[0], y[1], y[2], y[3]);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            mma_f16(s[u][b][0], q0[b].x, q0[b].y, q0[b].z, q0[b].w, x[0], x[1]);
            mma_f16(s[u][b][1], q0[b].x, q0[b].y, q0[b].z, q0[b].w, y[0], y[1]);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            mma_f16(s[u][b][0], q1[b].x, q1[b].y, q1[b].z, q1[b].w, x[2], x[3]);
            mma_f16(s[u][b][1], q1[b].x, q1[b].y, q1[b].z, q1[b].w, y[2], y[3]);
          }
        }
      }
    }
    // s[u][b][nt][e]: row g (e < 2) or g + 8 of block b, token 8 nt + 2t + (e & 1)
    uint32_t pa[NP][NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float &mA = m[b][0], &mB = m[b][1], p[NP][2][4], big = -INFINITY;
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const float scA = pg[u].ks * qsc[b][0], scB = pg[u].ks * qsc[b][1];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[u][nt][e] = fmaf(s[u][b][nt][e], e < 2 ? scA : scB, e < 2 ? -mA : -mB);
      }
      if constexpr (EDGE) {
        const int limA = last(b, 0), limB = last(b, 1);
#pragma unroll
        for (int u = 0; u < NP; ++u)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = 8 * nt + 2 * t + (e & 1);
              if (tok >= pg[u].nv || pg[u].pos0 + tok > (e < 2 ? limA : limB))
                p[u][nt][e] = -INFINITY;
            }
      }
#pragma unroll
      for (int u = 0; u < NP; ++u)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          big = fmaxf(big,
                      fmaxf(fmaxf(p[u][nt][0], p[u][nt][1]), fmaxf(p[u][nt][2], p[u][nt][3])));
      if (__any_sync(0xffffffffu, big > kSlack)) {
        float nA = kUnset, nB = kUnset;
#pragma unroll
        for (int u = 0; u < NP; ++u)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = s[u][b][nt][e] * (pg[u].ks * qsc[b][e >> 1]);
              float& x = p[u][nt][e];
              x = x == -INFINITY ? -INFINITY : y;
              if (e < 2) nA = fmaxf(nA, x);
              else nB = fmaxf(nB, x);
            }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          nA = fmaxf(nA, __shfl_xor_sync(0xffffffffu, nA, o));
          nB = fmaxf(nB, __shfl_xor_sync(0xffffffffu, nB, o));
        }
        nA = fmaxf(nA - kBelow, mA);
        nB = fmaxf(nB - kBelow, mB);
        const float aA = fast_exp2(mA - nA), aB = fast_exp2(mB - nB);
        mA = nA;
        mB = nB;
        l[b][0] *= aA;
        l[b][1] *= aB;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          acc[b][i][0] *= aA;
          acc[b][i][1] *= aA;
          acc[b][i][2] *= aB;
          acc[b][i][3] *= aB;
        }
#pragma unroll
        for (int u = 0; u < NP; ++u)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[u][nt][e] -= e < 2 ? nA : nB;
      }
#pragma unroll
      for (int u = 0; u < NP; ++u) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[u][nt][e] = fast_exp2(p[u][nt][e]);
        l[b][0] += (p[u][0][0] + p[u][0][1]) + (p[u][1][0] + p[u][1][1]);
        l[b][1] += (p[u][0][2] + p[u][0][3]) + (p[u][1][2] + p[u][1][3]);
        pa[u][b][0] = f32x2_to_f16x2(p[u][0][0], p[u][0][1]);
        pa[u][b][1] = f32x2_to_f16x2(p[u][0][2], p[u][0][3]);
        pa[u][b][2] = f32x2_to_f16x2(p[u][1][0], p[u][1][1]);
        pa[u][b][3] = f32x2_to_f16x2(p[u][1][2], p[u][1][3]);
      }
    }
    if constexpr (EDGE) {  // (as for 8 rows)
      const int page = exponent_field(pg[0].vs);
      if (!unit_fits(page, unit)) {
        const int to = unit_for(page, unit, largest);
        const float f = pow2_or_zero(unit - to);
        unit = to;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][i][e] *= f;
      }
    }
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const uint4 v0 = lds128_at<2 * kE2m1Tile>(pg[u].k16);
      const uint4 v1 = lds128_at<2 * kE2m1Tile + 512>(pg[u].k16);
      const uint32_t sw = lds32_at<2 * kE2m1Tile>(pg[u].k4);
      auto add = [&](uint32_t scales) {
        uint32_t slo, shi;  // scales of group g's tokens 2t, 2t + 1 and 2t + 8, 2t + 9
        e4m3x4_to_f16(scales, slo, shi);
        const uint32_t f = pow2_f16x2<EDGE>(exponent_field(pg[u].vs) - unit);
        slo = mul_f16x2(slo, f);
        shi = mul_f16x2(shi, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // column g of tiles 2i, 2i + 1: dims 16g + 2i, + 1
          uint32_t b00, b10, b01, b11;
          e2m1x8_scaled(w_of(i < 4 ? v0 : v1, i & 3), slo, shi, b00, b10, b01, b11);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t(&a)[4] = pa[u][b];
            mma_f16(acc[b][2 * i], a[0], a[1], a[2], a[3], b00, b01);
            mma_f16(acc[b][2 * i + 1], a[0], a[1], a[2], a[3], b10, b11);
          }
        }
      };
      if constexpr (!EDGE) {
        add(sw);
      } else {  // (as for 8 rows)
        uint32_t clean = sw & e2m1_token_mask(pg[u].nv, t);
        const int first = e2m1_first_nan(clean, t);  // of group g
        add(clean);
        if (__any_sync(0xffffffffu, first < 16)) {
          // columns 2t, 2t + 1 of every tile: groups 2t and 2t + 1
          const int f0 = __shfl_sync(0xffffffffu, first, 8 * t);
          const int f1 = __shfl_sync(0xffffffffu, first, 8 * t + 4);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int limA = last(b, 0) - pg[u].pos0, limB = last(b, 1) - pg[u].pos0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (f0 < 16 && f0 <= limA) acc[b][i][0] = __int_as_float(0x7FFFFFFF);
              if (f1 < 16 && f1 <= limA) acc[b][i][1] = __int_as_float(0x7FFFFFFF);
              if (f0 < 16 && f0 <= limB) acc[b][i][2] = __int_as_float(0x7FFFFFFF);
              if (f1 < 16 && f1 <= limB) acc[b][i][3] = __int_as_float(0x7FFFFFFF);
            }
          }
        }
      }
    }
  }
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) l[b][hr] += __shfl_xor_sync(0xffffffffu, l[b][hr], o);
        m[b][hr] = final_reference(m[b][hr], l[b][hr]);
      }
  }
};

template <int NB>
__global__ void __launch_bounds__(E2m1Cfg<NB>::THREADS, 1) e2m1_split_kernel(const DecodeArgs a) {
  using C = E2m1Cfg<NB>;
  constexpr bool WIDE = NB > 0;
  constexpr int D = 128, ST = C::ST;
  extern __shared__ __align__(1024) uint8_t smem[];
  int32_t* pfx_s = reinterpret_cast<int32_t*>(smem + C::OFF_PFX);
  int* wsum_s = reinterpret_cast<int*>(smem + C::OFF_WSUM);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int B = a.B, Hkv = a.d.num_kv_heads, Hs = a.Hs, HG = a.HG;
  // row blocks of a kv head, one a warp
  const int RBW = a.R8 / C::ROWS, Hv = Hs * RBW;
  if (Hs < 1 || RBW < 1 || (!WIDE && RBW != 1) || RBW * C::ROWS != a.R8 || a.R < 1 ||
      a.R > a.R8 || Hs * HG != Hkv || C::WARPS % Hv != 0 || a.sub != C::WARPS / Hv ||
      a.unit_tokens != 32 || (a.self_plan && B + 1 > kPfxCache)) {
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) set_error(a.d.ctl, KV_ERR_INTERNAL);  // host chose a bad configuration
    return;
  }
  pdl_wait();
  pdl_trigger();  // the combine's CTAs may wait resident in what this kernel leaves free
  const bool cached = B + 1 <= kPfxCache;
  if (a.self_plan) {
    const bool refused = decode_plan_shared(a, pfx_s, wsum_s);
    if (blockIdx.x == 0) decode_plan_store(a, pfx_s, refused);
  } else if (cached) {
    for (int i = threadIdx.x; i <= B; i += C::THREADS) pfx_s[i] = a.ws.pfx[i];
  }
  __syncthreads();  // the plan is visible to every warp
  const int32_t* pfx = cached ? pfx_s : a.ws.pfx;
  const long long total = (long long)pfx[B] * HG;
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long x_begin = (long long)blockIdx.x * per;
  const int n_units = (int)(min(total, x_begin + per) - x_begin);  // of this CTA
  if (n_units <= 0) return;
  const Cursor start = cursor_at(pfx, B, HG, x_begin);

  const int WPH = C::WARPS / Hv;                // warps per virtual head (kv head, row block)
  const int vh = warp % Hv, lg = warp / Hv;
  const int hw = vh / RBW, n0 = (vh - hw * RBW) * C::ROWS;  // kv head of the group, first query row
  const uint32_t ring = smem_u32(smem) + warp * (ST * kStage);
  UnitTable* table = reinterpret_cast<UnitTable*>(smem + C::OFF_UNIT) + warp;

  // ---- this warp's units: i = 0, 1, .. are the CTA's lg + WPH i, in batches of 16.
  // Lane l looks after page l % 2 of unit 16 b + l / 2: page ids are loaded two
  // batches ahead, scales one.
  const int count = (n_units - lg + WPH - 1) / WPH;  // (<= 0: none)
  struct Id {
    int p, hg;  // page id (-1: none; -2: out of range; -3: a stale tag), head group
  };
  struct Raw {
    int L, p, j, r, hg;  // length, page id as loaded, page number, request (-1: no unit)
  };
  auto locate = [&](int b) {
    const int i = 16 * b + (lane >> 1);
    Raw w{0, -1, 0, -1, 0};
    if (i < count) {
      const long long x = x_begin + lg + WPH * i;
      const Cursor c = cursor_at(pfx, B, HG, x);
      w.r = c.r;
      w.hg = c.h;
      w.j = 2 * (int)(x - c.seg_start) + (lane & 1);
      // (a unit's second page may lie behind the length; both loads at once)
      w.L = a.seq_lens[c.r];
      if (w.j < a.max_pages) w.p = a.page_table[(long long)c.r * a.max_pages + w.j];
    }
    return w;
  };
  auto check = [&](const Raw& w) {
    Id id{-1, w.hg};
    if (w.r < 0 || w.L <= 16 * w.j) return id;
    // the fused check: the tag is compared before the page is fetched
    id.p = w.p < 0 || w.p >= a.d.num_pages ? -2
           : a.exp_tags == nullptr ||
                   a.d.tags[w.p] == a.exp_tags[(long long)w.r * a.max_pages + w.j]
               ? w.p
               : -3;
    return id;
  };
  // batch b into the table, its tiles and then their scales
  auto fill_tiles = [&](int b, const Id& id) {
    if (id.p == -2) set_error(a.d.ctl, KV_ERR_BAD_PAGE_ID);
    const int tile = id.p < 0 ? -1 : id.p * Hkv + id.hg * Hs + hw;  // (2^31 tiles are 2 TB)
    reinterpret_cast<int*>(table->tile)[32 * (b & 1) + lane] = tile;
    return tile;
  };
  auto load_scales = [&](int tile) {
    float2 sc = make_float2(1.0f, 1.0f);
    if (tile >= 0) sc = make_float2(a.d.k_scale[tile], a.d.v_scale[tile]);
    // (V's is taken by its exponent alone: one that no append leaves, negative or not finite, makes
    // NaN of the page's scores instead)
    if (__float_as_uint(sc.y) >= 0x7F800000u) sc = make_float2(__int_as_float(0x7FFFFFFF), 1.0f);
    return sc;
  };
  auto fill_scales = [&](int b, float2 sc) {
    reinterpret_cast<float*>(table->ks)[32 * (b & 1) + lane] = sc.x;
    reinterpret_cast<float*>(table->vs)[32 * (b & 1) + lane] = sc.y;
  };
  // Unit i's copies into stage st: 16 bytes a lane each, a group a unit.
  const uint64_t policy = l2_evict_first_policy();
  // (WIDE, which is bound by its warps' instructions: where one of its pages is not there, or
  // must not be read, page 0's tile is copied: it is never counted, or its request gets no
  // output.  Without a branch the copies' addresses are worked out between what surrounds them.
  // Up to 8 rows, bound by HBM, it is 1 us in 128 the other way.)
  auto fetch = [&](int i, int st) {
    const int2 tl = table->tile[i & 31];
    if (i < count && (tl.x & tl.y) >= 0) {
      const uint32_t dst = ring + st * kStage + 16 * lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tile = k & 1 ? tl.y : tl.x;
        if (!WIDE && tile < 0) continue;
        const uint8_t* src = static_cast<const uint8_t*>(k < 2 ? a.d.k_cache : a.d.v_cache) +
                             (long long)max(tile, 0) * kE2m1Tile + 16 * lane;
        copy16(dst + k * kE2m1Tile, src, policy);
        copy16(dst + k * kE2m1Tile + 512, src + 512, policy);
        if (lane < 8) copy16(dst + k * kE2m1Tile + 1024, src + 1024, policy);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // a piece's queries into the L2: 256 bytes a row, two lanes
  auto prefetch_queries = [&](const Cursor& c) {
#pragma unroll
    for (int k = 0; k < (NB > 1 ? NB : 1); ++k) {
      const int row = n0 + 16 * k + (lane >> 1);
      if (row < a.R && (WIDE || lane < 16)) {
        const int tq = row / a.G, hq = (c.h * Hs + hw) * a.G + row - tq * a.G;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            a.q + (((long long)c.r * a.T + tq) * a.Hq + hq) * D + 64 * (lane & 1)));
      }
    }
  };
  prefetch_queries(start);
  // (the first units' pages are on their way before anything else is looked up)
  uint32_t bad_pages, bad_next;
  Raw ids;
  {
    const Id id0 = check(locate(0));
    const int t0 = fill_tiles(0, id0);
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < ST; ++i) fetch(i, i);
    const float2 s0 = load_scales(t0);
    const Raw w1 = locate(1);
    ids = locate(2);
    fill_scales(0, s0);
    const Id id1 = check(w1);
    fill_scales(1, load_scales(fill_tiles(1, id1)));
    bad_pages = __ballot_sync(0xffffffffu, id0.p < -1);
    bad_next = __ballot_sync(0xffffffffu, id1.p < -1);
    __syncwarp();
  }
  int batch = 0;

  Cursor seg = start;
  int done = 0;          // units of the CTA before this piece
  int i = 0, st = 0;  // the warp's next unit and its stage
  const int G = a.G, T = a.T, R = a.R;
  const float ssl = a.sm_scale_log2;

  while (done < n_units) {
    const int u0 = (int)(x_begin + done - seg.seg_start);  // the piece's first unit in its segment
    const int n_piece = min(seg.np - u0, n_units - done);
    const int r = seg.r, h = seg.h * Hs + hw, L = a.seq_lens[r];
    const int rel = done + n_piece - lg;
    const int i_end = rel > 0 ? (rel + WPH - 1) / WPH : 0;
    // units whose 32 positions every query token sees: below i_full
    const int see = max(0, L - T + 1) / 32 + done - u0 - lg;
    const int i_full = min(i_end, see > 0 ? (see + WPH - 1) / WPH : 0);
    int pos = 32 * (lg + WPH * i - done + u0);  // of unit i
    bool bad = false;

    auto units = [&](auto& rows) {
      auto unit = [&](auto whole) {
        // every lane's copies of the unit have landed
        asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
        __syncwarp();
        const float2 ks = table->ks[i & 31], vs = table->vs[i & 31];
        E2m1Page pg[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          pg[k].k16 = ring + st * kStage + k * kE2m1Tile + 16 * lane;
          pg[k].k4 = ring + st * kStage + k * kE2m1Tile + kE2m1Scales + 4 * lane;
          pg[k].ks = k ? ks.y : ks.x;
          pg[k].vs = k ? vs.y : vs.x;
          pg[k].pos0 = pos + 16 * k;
          pg[k].nv = min(16, L - pg[k].pos0);
        }
        pos = (int)((uint32_t)pos + 32u * WPH);  // (may pass 2^31 behind the last unit)
        if constexpr (decltype(whole)::value) {
          rows.template pages<2, false>(pg);
        } else {
          // (a page behind the length was not fetched)
#pragma unroll 1
          for (int k = 0; k < 2; ++k)
            if (k == 0 ? pg[0].nv > 0 : pg[1].nv > 0) {
              const E2m1Page one[1] = {k == 0 ? pg[0] : pg[1]};
              rows.template pages<1, true>(one);
            }
        }
        __syncwarp();  // every lane has read its part of the stage
        fetch(i + ST, st);
        ++i;
        if (++st == ST) st = 0;
      };
      while (i < i_end) {
        if ((i >> 4) != batch) {
          ++batch;
          bad_pages = bad_next;
          const Id id = check(ids);
          fill_scales(batch + 1, load_scales(fill_tiles(batch + 1, id)));
          bad_next = __ballot_sync(0xffffffffu, id.p < -1);
          __syncwarp();
          ids = locate(batch + 2);
        }
        // (a unit that must not be read may be computed on all the same: the
        // request gets no output)
        const int stop = min(i_end, 16 * batch + 16);
        bad = bad || (bad_pages >> (2 * (i & 15))) << (32 - 2 * (stop - i)) != 0;
        const int full_stop = min(stop, i_full);
        // Whether the whole units' pages fit the unit of the outputs, two at a time; the first unit
        // is one that most of them fit
        const int mine = (lane >> 1) + 16 * batch;
        const bool whole = mine >= i && mine < full_stop;
        const int page = exponent_field(reinterpret_cast<const float*>(table->vs)[32 * (batch & 1) + lane]);
        if (rows.unit < 0) {
          rows.largest = (int)__reduce_max_sync(0xffffffffu, whole ? page : 0);
          if (rows.largest == 0) rows.largest = exponent_field(table->vs[i & 31].x);
          rows.unit = rows.largest - (kOver - 2);
        }
        const int fast =
            __any_sync(0xffffffffu, whole && !unit_fits(page, rows.unit)) ? i : full_stop;
        while (i < fast) unit(TrueType{});
        while (i < stop) unit(FalseType{});
      }
    };

    if (done + n_piece < n_units) {
      Cursor next = seg;
      cursor_next(next, pfx, B, HG);
      prefetch_queries(next);
    }
    // this warp's partial of the piece
    const long long prow =
        ((((long long)r * HG + seg.h + blockIdx.x) * a.sub + lg) * Hs + hw) * a.R8 + n0;
    float* ml = a.ws.ml_part + prow * 2;
    float* op = a.ws.o_part + prow * D;
    if constexpr (WIDE) {
      // ---- Q as A operands {a0, a1, a2, a3} of k-step j = rows g, g + 8 x dims
      // d(j) + 0, 1 and d(j) + 2, 3 with d(j) = 16t + 4j (j < 4), 64 + 16t + 4 (j - 4)
      uint32_t* qs = reinterpret_cast<uint32_t*>(smem + C::OFF_Q + warp * C::QBYTES);
      float qsc[NB][2];  // score scales of rows g and g + 8 of a block, with the row's 2^-e
      __syncwarp();      // the last piece's reads
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t qa[8][4];
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const int row = n0 + 16 * b + g + 8 * hr;
          const bool live = row < R;
          const int tq = live ? row / G : 0, hq = live ? h * G + row % G : 0;
          const uint16_t* qrow = a.q + (((long long)r * T + tq) * a.Hq + hq) * D + 16 * t;
          uint4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            v[u] = live ? *reinterpret_cast<const uint4*>(qrow + 8 * (u & 1) + 64 * (u >> 1))
                        : make_uint4(0, 0, 0, 0);
          uint32_t mb = max(max(bf16_absbits_max8(v[0]), bf16_absbits_max8(v[1])),
                            max(bf16_absbits_max8(v[2]), bf16_absbits_max8(v[3])));
          mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
          mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
          const int e = q_row_exp(mb);
          const float pw = pow2f(e);
          qsc[b][hr] = row_score_scale(ssl, e, mb);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            qa[2 * u][hr] = bf16x2_to_f16x2_scaled(v[u].x, pw);
            qa[2 * u][2 + hr] = bf16x2_to_f16x2_scaled(v[u].y, pw);
            qa[2 * u + 1][hr] = bf16x2_to_f16x2_scaled(v[u].z, pw);
            qa[2 * u + 1][2 + hr] = bf16x2_to_f16x2_scaled(v[u].w, pw);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(qs + ((8 * b + j) * 32 + lane) * 4) =
              make_uint4(qa[j][0], qa[j][1], qa[j][2], qa[j][3]);
      }
      __syncwarp();
      float m[NB][2], l[NB][2], acc[NB][16][4];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        m[b][0] = m[b][1] = kUnset;
        l[b][0] = l[b][1] = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          acc[b][k][0] = acc[b][k][1] = acc[b][k][2] = acc[b][k][3] = 0.0f;
      }
      E2m1Rows16<NB> rows{m, l, acc, smem_u32(qs) + 16 * lane, qsc, n0, G, T, L - T};
      units(rows);
      rows.finish();
      const int x = rows.unit < 0 ? 0 : rows.unit - 127;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const int down = partial_shift(x, m[b][hr], l[b][hr]);
          if (t == 0)
            *reinterpret_cast<float2*>(ml + 2 * (16 * b + g + 8 * hr)) =
                make_float2(m[b][hr] + down, bad ? -1.0f : l[b][hr] * pow2f(-down));
          if (down != x) {
            const float f = pow2f(x - down);
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[b][k][2 * hr] *= f, acc[b][k][2 * hr + 1] *= f;
          }
        }
      // column c of tile k is dim 16 c + k: a lane's 32 dims of a row are contiguous
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4*>(op + (16 * b + g + 8 * (e >> 1)) * D + 32 * t +
                                       16 * (e & 1) + k) =
                make_float4(acc[b][k][e], acc[b][k + 1][e], acc[b][k + 2][e], acc[b][k + 3][e]);
    } else {
      // ---- query fragments of row g (zero for padding rows) in shared memory, those of
      // k-steps 2w and 2w + 1 a 16-byte word: k-step j has dims 16 (t + 4 (j / 4)) + 4 (j % 4) ..
      uint32_t* qs = reinterpret_cast<uint32_t*>(smem + C::OFF_Q + warp * C::QBYTES);
      float qsc0, qsc1;  // score scales of rows 2t, 2t + 1, with the row's 2^-e
      {
        const bool live = g < R;
        const int tq = live ? g / G : 0, hq = live ? h * G + g % G : 0;
        const uint16_t* qrow = a.q + (((long long)r * T + tq) * a.Hq + hq) * D + 16 * t;
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[u] = live ? *reinterpret_cast<const uint4*>(qrow + 8 * (u & 1) + 64 * (u >> 1))
                      : make_uint4(0, 0, 0, 0);
        uint32_t mb = max(max(bf16_absbits_max8(v[0]), bf16_absbits_max8(v[1])),
                          max(bf16_absbits_max8(v[2]), bf16_absbits_max8(v[3])));
        mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
        mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
        const int e = q_row_exp(mb);
        const float pw = pow2f(e);
        // rows 2t and 2t + 1 are held by the lanes g = 2t and 2t + 1
        const float sc = row_score_scale(ssl, e, mb);
        qsc0 = __shfl_sync(0xffffffffu, sc, 8 * t);
        qsc1 = __shfl_sync(0xffffffffu, sc, 8 * t + 4);
        __syncwarp();  // the last piece's reads
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(qs + (u * 32 + lane) * 4) =
              make_uint4(bf16x2_to_f16x2_scaled(v[u].x, pw), bf16x2_to_f16x2_scaled(v[u].y, pw),
                         bf16x2_to_f16x2_scaled(v[u].z, pw), bf16x2_to_f16x2_scaled(v[u].w, pw));
        __syncwarp();
      }
      float m0 = kUnset, m1 = kUnset, l0 = 0.0f, l1 = 0.0f;
      float acc[8][4];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.0f;
      E2m1Rows8 rows{m0, m1, l0, l1, acc, smem_u32(qs) + 16 * lane, qsc0, qsc1, G, T, L - T};
      units(rows);
      rows.finish();
      const int x = rows.unit < 0 ? 0 : rows.unit - 127;
      const int down0 = partial_shift(x, m0, l0), down1 = partial_shift(x, m1, l1);
      if (down0 != x || down1 != x) {
        const float f0 = pow2f(x - down0), f1 = pow2f(x - down1);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          acc[k][0] *= f0;
          acc[k][1] *= f1;
          acc[k][2] *= f0;
          acc[k][3] *= f1;
        }
      }
      if (g == 0)
        *reinterpret_cast<float4*>(ml + 4 * t) =
            make_float4(m0 + down0, bad ? -1.0f : l0 * pow2f(-down0), m1 + down1,
                        bad ? -1.0f : l1 * pow2f(-down1));
      // rows g, g + 8 of tile k are dims 16g + 2k, + 1: 16 contiguous dims of a row
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < 8; k += 2)
          *reinterpret_cast<float4*>(op + (2 * t + e) * D + 16 * g + 2 * k) =
              make_float4(acc[k][e], acc[k][e + 2], acc[k + 1][e], acc[k + 1][e + 2]);
    }
    done += n_piece;
    if (u0 + n_piece == seg.np) cursor_next(seg, pfx, B, HG);
  }
}

// ------------------------------------------------- combine

// O = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c over a segment's partials c: S
// warps an output row, S about a fourth to an eighth of the partials of a row, so that a
// warp's loads are in flight together and the kernel is a few round trips; lane l has
// dims 4l .. 4l + 3.  W: warps a block.
template <int W>
__global__ void __launch_bounds__(W * 32, W == 8 ? 4 : 1)
    e2m1_combine_kernel(const DecodeArgs a, int S) {
  constexpr int D = 128, kU = 8;  // partials loaded together
  __shared__ float4 st_o[W][32];
  __shared__ float2 st_ml[W];
  __shared__ int st_bad[W];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp & (S - 1);
  const int Hkv = a.d.num_kv_heads, R = a.R;
  const long long item = (long long)blockIdx.x * (W / S) + warp / S;
  const bool live = item < (long long)a.B * Hkv * R;
  // every warp reaches the block's barrier: no early return
  int r = 0, h = 0, n = 0, parts = 0;
  long long row0 = 0;
  bool skip = true;
  if (live) {
    const int rh = (int)(item / R);
    n = (int)(item - (long long)rh * R);
    r = rh / Hkv;
    h = rh - r * Hkv;
    const int first = a.ws.pfx[r], np = a.ws.pfx[r + 1] - first, all = a.ws.pfx[a.B];
    skip = a.ws.rq_skip[r];  // aborted or invalid length: output left untouched
    if (!skip && np > 0) {
      const int hg = h / a.Hs, hw = h - hg * a.Hs;
      const long long total = (long long)all * a.HG;
      const long long start = (long long)first * a.HG + (long long)hg * np, last = start + np - 1;
      int c0, c1;  // the CTAs whose ranges meet the segment
      if (total < (1ll << 31)) {
        const uint32_t per = ((uint32_t)total + a.grid - 1) / a.grid;
        c0 = (uint32_t)start / per;
        c1 = (uint32_t)last / per;
      } else {
        const long long per = (total + a.grid - 1) / a.grid;
        c0 = (int)(start / per);
        c1 = (int)(last / per);
      }
      parts = (c1 - c0 + 1) * a.sub;
      row0 = ((((long long)r * a.HG + hg + c0) * a.sub) * a.Hs + hw) * a.R8 + n;
    }
  }
  const int stride = a.Hs * a.R8;  // rows from a partial to the next
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float M = -INFINITY, L = 0.0f;
  bool bad = false;
  const int cnt = (parts - sub + S - 1) / S;  // this warp's: sub, sub + S, ..
  for (int j0 = 0; j0 < cnt; j0 += 32) {
    const int nj = min(32, cnt - j0);
    auto row_of = [&](int j) { return row0 + (long long)(sub + S * (j0 + j)) * stride; };
    auto load = [&](int j) {
      return j < nj ? *reinterpret_cast<const float4*>(a.ws.o_part + row_of(j) * D + 4 * lane)
                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    float4 o[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) o[u] = load(u);
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < nj) ml = *reinterpret_cast<const float2*>(a.ws.ml_part + row_of(lane) * 2);
    bad = bad || __any_sync(0xffffffffu, ml.y < 0.0f);
    const float Mc = warp_max(ml.x);
    if (Mc == -INFINITY) continue;  // nothing visible
    const float Mn = fmaxf(M, Mc), keep = exp2f(M - Mn);
    const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - Mn);
    L = L * keep + warp_sum(ml.y * w);
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
    for (int k = 0; k < nj; k += kU) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, (k + u) & 31);
        // (a partial that saw nothing is zeros; one whose weight is 0 may hold a V that is NaN)
        if (k + u < nj) {
          acc.x = fmaf(o[u].x, wu, acc.x);
          acc.y = fmaf(o[u].y, wu, acc.y);
          acc.z = fmaf(o[u].z, wu, acc.z);
          acc.w = fmaf(o[u].w, wu, acc.w);
        }
      }
      if (k + kU < nj)
#pragma unroll
        for (int u = 0; u < kU; ++u) o[u] = load(k + kU + u);
    }
    M = Mn;
  }
  if (S > 1) {
    st_o[warp][lane] = acc;
    if (lane == 0) {
      st_ml[warp] = make_float2(M, L);
      st_bad[warp] = bad;
    }
    __syncthreads();
    if (sub == 0) {
      // lane k: the state of the row's warp k (S <= 32); then the weighted outputs, independent
      const int k = warp + min(lane, S - 1);
      const float2 ml = lane < S ? st_ml[k] : make_float2(-INFINITY, 0.0f);
      bad = __any_sync(0xffffffffu, lane < S && st_bad[k] != 0);
      M = warp_max(ml.x);
      const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M);
      L = warp_sum(ml.y * w);
      acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int j = 0; j < S; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const float4 v = st_o[warp + j][lane];
        acc.x = fmaf(v.x, wj, acc.x);
        acc.y = fmaf(v.y, wj, acc.y);
        acc.z = fmaf(v.z, wj, acc.z);
        acc.w = fmaf(v.w, wj, acc.w);
      }
    }
  }
  if (!live || sub != 0) return;
  // fused tag check: the warp of the request's first row writes its abort bit
  // (every segment and row of a request meets the same pages)
  if (a.abort_out != nullptr && h == 0 && n == 0) a.abort_out[r] = (skip || bad) ? 1 : 0;
  if (skip || bad) return;
  const float inv = M == -INFINITY ? 0.0f : 1.0f / L;  // nothing visible: zeros
  uint2 w;
  w.x = f32x2_to_bf16x2(acc.x * inv, acc.y * inv);
  w.y = f32x2_to_bf16x2(acc.z * inv, acc.w * inv);
  const int tq = n / a.G, hq = h * a.G + n - tq * a.G;
  *reinterpret_cast<uint2*>(a.out + (((long long)r * a.T + tq) * a.Hq + hq) * D + 4 * lane) = w;
}

}  // namespace

int e2m1_split_warps(int kind) {
  return kind == kGqaE2m1Rows32   ? E2m1Cfg<2>::WARPS
         : kind == kGqaE2m1Rows16 ? E2m1Cfg<1>::WARPS
                                  : E2m1Cfg<0>::WARPS;
}

// What a piece costs beside its units (its queries, its first and last pages, its partial) in
// units, by which a request is counted longer.  Above 8 rows 12: 88 us against 100 without for 24
// requests of 4 drafts, 70 against 79 for the ragged batch above (6: 93 and 73, 20: 90 and 72).
// Up to 8 rows 4: 1 us in 128, where 16 takes it back.
int e2m1_unit_extra(int kind) { return kind == kGqaE2m1 ? 4 : 12; }

int e2m1_split_ctas_per_sm(int kind) {
  static int cache[64][3];  // by device, as the attribute below is; 0: not asked yet
  const int nb = kind - kGqaE2m1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cache[dev][nb] > 0) return cache[dev][nb];
  const auto kernel = nb == 2   ? e2m1_split_kernel<2>
                      : nb == 1 ? e2m1_split_kernel<1>
                                : e2m1_split_kernel<0>;
  const int smem = nb == 2 ? E2m1Cfg<2>::SMEM : nb == 1 ? E2m1Cfg<1>::SMEM : E2m1Cfg<0>::SMEM;
  int n = 0;
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      &n, kernel, 32 * e2m1_split_warps(kind), smem);
  if (e != cudaSuccess || n <= 0) return 0;
  cache[dev][nb] = n;
  return n;
}

namespace {

template <int NB>
cudaError_t launch_split(const DecodeArgs& a, cudaStream_t s) {
  return launch_pdl(e2m1_split_kernel<NB>, dim3(a.grid), dim3(E2m1Cfg<NB>::THREADS),
                    E2m1Cfg<NB>::SMEM, s, a);
}

}  // namespace

cudaError_t launch_e2m1_split(const DecodeArgs& a, int kind, cudaStream_t s, int* launches) {
  const cudaError_t e = kind == kGqaE2m1Rows32   ? launch_split<2>(a, s)
                        : kind == kGqaE2m1Rows16 ? launch_split<1>(a, s)
                                                 : launch_split<0>(a, s);
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_e2m1_combine(const DecodeArgs& a, cudaStream_t s, int* launches) {
  const long long rows = (long long)a.B * a.d.num_kv_heads * a.R;
  if (rows <= 0) return cudaSuccess;
  const double parts = a.sub * (1.0 + (double)a.grid / ((double)a.B * a.HG));  // a row, about
  int S = 1;
  while (S < 8 && 8.0 * S < parts) S *= 2;
  // (32 where the rows' blocks are one wave: 64 rows of 300 partials 40 us against 44 in all; 256
  // rows of 160, two waves, 36 against 32)
  if (parts > 128.0 && rows <= a.grid) S = 32;
  const int W = S == 32 ? 32 : 8;
  const long long blocks = (rows + W / S - 1) / (W / S);
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      launch_pdl(S == 32 ? e2m1_combine_kernel<32> : e2m1_combine_kernel<8>,
                 dim3((unsigned)blocks), dim3(W * 32), 0, s, a, S);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
