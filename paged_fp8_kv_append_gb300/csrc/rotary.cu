// rotary.cu -- kv_append_rotary: queries and keys rotated by their positions
// on one or several axes (a token's time, height and width), the keys and
// values quantised as they are written into the paged cache.
//
// Pair i of a head turns by a_i = position[axis(i)] * inv_freq[i]:
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a),
// the pair being dims (i, i + rot/2), or (2i, 2i + 1) when interleaved; dims
// from rot on pass through.  A position times a frequency is wanted as a
// fraction of a turn, which fp32 does not keep for a far position: the tables
// hold a frequency as turns * 2^64, and the 64-bit integer product drops the
// whole turns by itself and leaves the fraction, off by no more than position
// times the table's own rounding (fp64: 2^-55 turns for a frequency of 1), with
// two integer multiply-adds where fp64 (scarce here) would take six operations.
// Sine and cosine of the fraction are fp32.  A rotated key
// stays in fp32 until its one rounding: to e4m3 by its page's scale (amax/448
// of the page's rotated rows, as kv_append_quantize takes it of the rows it is
// given), or to bf16.
//
// Two launches: the append's plan kernel (append.cu: pages popped, tags
// stamped, lengths advanced), then this kernel, one CTA of 8 warps per
// (request, touched page): the angles of the page's tokens are computed once
// into shared memory and serve every query and key head of those tokens.  With
// few pages the heads are split over up to 8 CTAs, to about two an SM.
//
// Bounded by HBM for prompts (every value read and written once).  8 prompts
// of 1k-4k tokens, 64 query and 8 kv heads: 160 us with the plan, 5.3 TB/s of
// the 6.8 of a plain copy; queries alone run at 6.3 (their threads keep a
// token's sines in registers and have 8 loads of 16 bytes in flight), the
// rest is the quantising of keys and values, half of the instructions.  Two
// CTAs an SM at 128 registers: three at 80 spill and take 192 us; 4 of half
// the threads 179; prefetching a page's rows into L2 changes nothing; a split
// of the heads into 8 for all sizes 217.  One row a request (a decode step of
// 64) is bounded by latency: about 13 us for the two kernels in a graph, a chain of dependent
// loads each.  Other shapes take the slower tiles, whose values are stored element by element
// and whose keys are read twice: pages of 16 x 64 run at 3.4 TB/s, of 8 x 256 at 2.2.
//
// kv_append_norm_rotary normalises the heads in the same pass.  A row's sum of squares runs over
// the eight lanes that hold it (heads of 128).  The same prompts: 162 us (the bytes are the same:
// 122 at a plain copy's rate), of which the plan 9; the first query loads wait behind the page's
// angles no more (164 us against 169 in one run), the keys' and values' still do behind the queries.
#include "append_tile.cuh"
#include "common.cuh"
#include "e2m1.cuh"
#include "internal.h"
#include "quant.cuh"
#include "ragged.cuh"

namespace kvfp8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAhead = 4;   // query units a thread has in flight
constexpr int kDepth = 6;  // the same where they come through shared memory

// A frequency as the table holds it: turns per position in units of 2^-64,
// whole turns dropped.
struct Freq {
  long long turns;
  int axis;    // -1: the tables name an axis that positions does not have
  float skew;  // 0, or NaN for a frequency that is not finite
};
static_assert(sizeof(Freq) == 16, "one shared load");

// A unit is two 8-value chunks of a row, 8 pairs: chunks j and j + rot/16 for
// j < rot/16 (pair k of dims k and k + rot/2: value k of each; neighbouring
// pairs: 4 in each chunk), and the rest of the row in the same way, so that
// the lanes of a row load and store neighbouring chunks.
struct UnitPlace {
  int c0, c1;  // chunk numbers
  bool turn;
};
__device__ __forceinline__ UnitPlace unit_place(int j, int rot16, int upr) {
  UnitPlace u;
  u.turn = j < rot16;
  u.c0 = u.turn ? j : j + rot16;
  u.c1 = u.c0 + (u.turn ? rot16 : upr - rot16);
  return u;
}

// Where 16 bytes (two pairs' sines and cosines) of a token's row lie in it.  Neighbouring units
// read 64 bytes each, and in order eight of them meet in two groups of banks: where every head's
// unit reads them anew (NORM) they are spread; elsewhere the addresses would cost registers.
template <bool NORM>
__device__ __forceinline__ int angle_chunk(int k) {
  return NORM ? (k & ~3) | ((k ^ (k >> 3)) & 3) : k;
}

// (cos, sin) of a unit's 8 pairs from its token's row of them
template <bool IL, bool NORM>
__device__ __forceinline__ void unit_angles(const float2* row, int j, int rot16, float2 (&c)[8]) {
  const float4* a = reinterpret_cast<const float4*>(row + (NORM ? 0 : (IL ? 4 : 8) * j));
  const float4* b = NORM ? a : IL ? reinterpret_cast<const float4*>(row + 4 * (j + rot16)) : a + 2;
  const int k0 = NORM ? (IL ? 2 : 4) * j : 0, k1 = NORM ? (IL ? 2 * (j + rot16) : k0 + 2) : 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float4 t = k < 2 ? a[angle_chunk<NORM>(k0 + k)] : b[angle_chunk<NORM>(k1 + k - 2)];
    if (NORM) t = make_float4(t.x, t.z, t.y, t.w);  // (as they lie there: two cosines, two sines)
    c[2 * k] = make_float2(t.x, t.y);
    c[2 * k + 1] = make_float2(t.z, t.w);
  }
}

// A head's norm: y = x / sqrt(mean(x^2) + eps) * weight, as a thread applies it to its unit.
// The sum runs over the upr neighbouring lanes of the row (a power of two), in fp32.
struct UnitNorm {
  const uint4 *w0, *w1;  // bf16 weights of the chunks c0 and c1 (read at each use: they stay in
                         // the L1, and registers are what a key page lacks)
  float eps, inv_d;
  uint32_t lanes;  // the row's lanes
  int upr;
  bool on;
};
template <bool NORM>
__device__ __forceinline__ UnitNorm unit_norm(const uint16_t* weight, float eps, int D,
                                              const UnitPlace& p) {
  UnitNorm n;
  n.on = NORM && weight != nullptr;
  if (!n.on) return n;
  n.w0 = reinterpret_cast<const uint4*>(weight) + p.c0;
  n.w1 = reinterpret_cast<const uint4*>(weight) + p.c1;
  n.eps = eps;
  n.inv_d = 1.0f / D;  // exact
  n.upr = D / 16;
  const int lane = threadIdx.x & 31;
  n.lanes = (uint32_t)((1ull << n.upr) - 1) << (lane & ~(n.upr - 1));
  return n;
}

// The unit's values normalised (NORM) and rotated: x[0..7] of chunk c0, x[8..15] of c1.
template <bool IL, bool NORM>
__device__ __forceinline__ void unit_turn(uint4 a, uint4 b, bool turn, const float2 (&c)[8],
                                          const UnitNorm& n, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
  }
  if (NORM && n.on) {
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) ss = fmaf(x[k], x[k], ss);
    for (int o = 1; o < n.upr; o <<= 1) ss += __shfl_xor_sync(n.lanes, ss, o);
    const float r = rsqrtf(fmaf(ss, n.inv_d, n.eps));
    const uint4 w0 = __ldg(n.w0), w1 = __ldg(n.w1);
    const uint32_t g[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[2 * k] = x[2 * k] * r * bf16_lo(g[k]);
      x[2 * k + 1] = x[2 * k + 1] * r * bf16_hi(g[k]);
    }
  }
  if (!turn) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float& p = IL ? x[2 * k] : x[k];
    float& q = IL ? x[2 * k + 1] : x[8 + k];
    const float p0 = p, q0 = q;
    p = p0 * c[k].x - q0 * c[k].y;
    q = q0 * c[k].x + p0 * c[k].y;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 pack8_bf16(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// 8 codes of x / s, as the append kernels divide
__device__ __forceinline__ uint2 codes8(const float* x, float s, float rs) {
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = e4m3x2(div_by_scale(x[2 * k], s, rs), div_by_scale(x[2 * k + 1], s, rs));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// where |x| <= 448 s and scale_fast_ok(s): the quotient by one corrected product
__device__ __forceinline__ uint2 codes8_fresh(const float* x, float s, float rs) {
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = e4m3x2(div_fresh(x[2 * k], s, rs), div_fresh(x[2 * k + 1], s, rs));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// A thread's slots in shared memory for normalised heads of 128: 32 bytes each, 16 of a unit's
// first chunk and 16 of its second.
constexpr uint32_t kHalfSlot = 16 * kThreads, kSlot = 2 * kHalfSlot;
__device__ __forceinline__ void copy16(uint32_t dst_smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst_smem), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 take16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// One (page, kv head) key tile by one warp: `nrows` rows from slot0 on; any
// shape, page and scale, a unit at a time (kept out of line: a fresh page's
// code stays small, and nothing of it lives across this call).
template <bool IL, bool NORM>
__device__ __noinline__ void key_tile_any(const uint16_t* src, long long stride, int nrows, int D,
                                          int rot16, const float2* cs, const uint16_t* weight,
                                          float eps, bool fp8, bool fresh,
                                          bool requant, float* scale_slot, uint8_t* dst,
                                          int slot0) {
  const int lane = threadIdx.x & 31, upr = D / 16, total = nrows * upr;
  float s = 1.0f, m = 0.0f;
  // pass 0 finds the scale, pass 1 writes
#pragma unroll 1
  for (int pass = fp8 && (fresh || requant) ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1 && fp8) {
      if (fresh) {
        s = scale_from_amax(warp_max(m));
        if (lane == 0) *scale_slot = s;
      } else {
        s = *scale_slot;
        const float s_new = requant ? scale_from_amax(warp_max(m)) : s;
        if (s_new > s) {  // a larger scale for the new rows: re-encode the old ones
          requant_block(dst, slot0, D, false, 0, s, s_new, lane, 32);
          __syncwarp();
          if (lane == 0) *scale_slot = s_new;
          s = s_new;
        }
      }
    }
    const float rs = __frcp_rn(s);
#pragma unroll 1
    for (int u = lane; u < total; u += 32) {  // (whole rows: total is a multiple of upr)
      const int i = u / upr, j = u - i * upr;
      const UnitPlace p = unit_place(j, rot16, upr);
      const uint4* row = reinterpret_cast<const uint4*>(src + i * stride);
      float2 c[8];
      float x[16];
      if (p.turn) unit_angles<IL, NORM>(cs + i * rot16 * 8, j, rot16, c);
      unit_turn<IL, NORM>(row[p.c0], row[p.c1], p.turn, c, unit_norm<NORM>(weight, eps, D, p), x);
      if (pass == 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
        continue;
      }
      const long long at = (long long)(slot0 + i) * D;
      if (fp8) {
        uint2* o = reinterpret_cast<uint2*>(dst + at);
        o[p.c0] = codes8(x, s, rs);
        o[p.c1] = codes8(x + 8, s, rs);
      } else {
        uint4* o = reinterpret_cast<uint4*>(dst + 2 * at);
        o[p.c0] = pack8_bf16(x);
        o[p.c1] = pack8_bf16(x + 8);
      }
    }
  }
}

// The same for a whole fresh page of 16 x 128 keys: its loads are issued
// together and its turned values stay in registers.
template <bool IL>
__device__ __forceinline__ void key_page_16x128(const uint16_t* src, long long stride, int rot16,
                                                const float2* cs, bool fp8, float* scale_slot,
                                                uint8_t* dst) {
  const int lane = threadIdx.x & 31, j = lane & 7, i0 = lane >> 3;  // rows i0 + 4 k
  const UnitPlace p = unit_place(j, rot16, 8);
  uint4 raw[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4* row = reinterpret_cast<const uint4*>(src + (i0 + 4 * k) * stride);
    raw[k][0] = __ldcs(row + p.c0);
    raw[k][1] = __ldcs(row + p.c1);
  }
  const UnitNorm none = unit_norm<false>(nullptr, 0.0f, 128, p);
  float x[4][16];
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 c[8];
    if (p.turn) unit_angles<IL, false>(cs + (i0 + 4 * k) * rot16 * 8, j, rot16, c);
    unit_turn<IL, false>(raw[k][0], raw[k][1], p.turn, c, none, x[k]);
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[k][e]));
  }
  if (!fp8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint4* o = reinterpret_cast<uint4*>(dst + (i0 + 4 * k) * 256);
      o[p.c0] = pack8_bf16(x[k]);
      o[p.c1] = pack8_bf16(x[k] + 8);
    }
    return;
  }
  const float s = scale_from_amax(warp_max(m)), rs = __frcp_rn(s);
  if (!scale_fast_ok(s)) {
    key_tile_any<IL, false>(src, stride, 16, 128, rot16, cs, nullptr, 0.0f, true, true, false,
                            scale_slot, dst, 0);
    return;
  }
  if (lane == 0) *scale_slot = s;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint2* o = reinterpret_cast<uint2*>(dst + (i0 + 4 * k) * 128);
    o[p.c0] = codes8_fresh(x[k], s, rs);
    o[p.c1] = codes8_fresh(x[k] + 8, s, rs);
  }
}

// The same of keys that are normalised too: with the weights their values do not fit the
// registers, and what spills finds little of the L1 beside the queries' slots (180 us for 8
// prompts became 205 with more of either).  So the rows wait in the thread's slots, and are
// normalised and turned once for the scale and once for the codes (172 us).
template <bool IL>
__device__ __noinline__ void key_page_norm_16x128(const uint16_t* src, long long stride, int rot16,
                                                  const float2* cs, uint32_t slots,
                                                  const uint16_t* weight, float eps, bool fp8,
                                                  float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, j = lane & 7, i0 = lane >> 3;  // rows i0 + 4 k
  const UnitPlace p = unit_place(j, rot16, 8);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4* row = reinterpret_cast<const uint4*>(src + (i0 + 4 * k) * stride);
    copy16(slots + k * kSlot, row + p.c0);
    copy16(slots + k * kSlot + kHalfSlot, row + p.c1);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  const UnitNorm norm = unit_norm<true>(weight, eps, 128, p);
  auto turned = [&](int k, float (&y)[16]) {
    float2 c[8];
    if (p.turn) unit_angles<IL, true>(cs + (i0 + 4 * k) * rot16 * 8, j, rot16, c);
    unit_turn<IL, true>(take16(slots + k * kSlot), take16(slots + k * kSlot + kHalfSlot), p.turn, c,
                        norm, y);
  };
  float m = 0.0f;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    float y[16];
    turned(k, y);
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(y[e]));
    if (!fp8) {
      uint4* o = reinterpret_cast<uint4*>(dst + (i0 + 4 * k) * 256);
      o[p.c0] = pack8_bf16(y);
      o[p.c1] = pack8_bf16(y + 8);
    }
  }
  if (!fp8) return;
  const float s = scale_from_amax(warp_max(m)), rs = __frcp_rn(s);
  if (lane == 0) *scale_slot = s;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    float y[16];
    turned(k, y);
    uint2* o = reinterpret_cast<uint2*>(dst + (i0 + 4 * k) * 128);
    if (scale_fast_ok(s)) {
      o[p.c0] = codes8_fresh(y, s, rs);
      o[p.c1] = codes8_fresh(y + 8, s, rs);
    } else {
      o[p.c0] = codes8(y, s, rs);
      o[p.c1] = codes8(y + 8, s, rs);
    }
  }
}

// The keys of a 4-bit tile (e2m1.cuh), from their fp32 values: up to 16 rows from slot0 on, lane
// (i, j) with unit j of rows i, i + 4, ..  A group's 16 dims are two chunks, the other of which
// may be another lane's.
template <bool IL, bool NORM>
__device__ __noinline__ void key_tile_e2m1(const uint16_t* src, long long stride, int nrows,
                                           int slot0, int rot16, const float2* cs,
                                           const uint16_t* weight, float eps, bool fresh,
                                           float* scale_slot, uint8_t* dst) {
  const int lane = threadIdx.x & 31, j = lane & 7, i0 = lane >> 3;
  const UnitPlace p = unit_place(j, rot16, 8);
  const UnitNorm norm = unit_norm<NORM>(weight, eps, 128, p);
  // the unit of chunk c, and 8 where it is the unit's second chunk
  auto unit_of = [&](int c) {
    return c < rot16 ? c : c < 2 * rot16 ? c - rot16 + 8 : c < 8 + rot16 ? c - rot16 : c;
  };
  const int other0 = unit_of(p.c0 ^ 1), other1 = unit_of(p.c1 ^ 1);
  float x[4][16], m[4][2], block = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = i0 + 4 * k;
    const bool ok = i < nrows;
    const uint4* row = reinterpret_cast<const uint4*>(src + (ok ? i : 0) * stride);
    float2 c[8];
    if (p.turn) unit_angles<IL, NORM>(cs + (ok ? i : 0) * rot16 * 8, j, rot16, c);
    unit_turn<IL, NORM>(row[p.c0], row[p.c1], p.turn, c, norm, x[k]);
    uint32_t b[2] = {0, 0};  // bit patterns: a NaN is the largest
#pragma unroll
    for (int e = 0; e < 16; ++e)
      b[e >> 3] = max(b[e >> 3], __float_as_uint(x[k][e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = (h ? other1 : other0) & 7, second = (h ? other1 : other0) & 8;
      const uint32_t b0 = __shfl_sync(0xffffffffu, b[0], (lane & 24) | o);
      const uint32_t b1 = __shfl_sync(0xffffffffu, b[1], (lane & 24) | o);
      m[k][h] = __uint_as_float(max(b[h], second ? b1 : b0));
      if (ok) block = fmaxf(block, finite_or_zero(m[k][h]));
    }
  }
  const float inv_s = pow2_inverse(e2m1_tile_scale(block, fresh, scale_slot));
  const int chunk[2] = {p.c0, p.c1};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int slot = slot0 + i0 + 4 * k;
    if (i0 + 4 * k >= nrows) continue;
    float f[2];
    const uint32_t sc = e2m1_group_scales(m[k][0], m[k][1], inv_s * kE2m1Sixth, inv_s, f[0], f[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = chunk[h] >> 1;
      const uint64_t ff = pack2(f[h], f[h]);
      uint64_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = mul2(pack2(x[k][8 * h + 2 * e], x[k][8 * h + 2 * e + 1]), ff);
      *reinterpret_cast<uint32_t*>(dst + 64 * slot + 16 * (g & 3) + 8 * (g >> 2) +
                                   4 * (chunk[h] & 1)) = e2m1x8(v[0], v[1], v[2], v[3]);
      if ((chunk[h] & 1) == 0)
        dst[kE2m1Scales + 16 * (slot & 7) + 4 * (g & 3) + 2 * (slot >> 3) + (g >> 2)] =
            (uint8_t)(sc >> (8 * h));
    }
  }
}
__device__ __noinline__ void value_tile_e2m1(const uint16_t* src, long long stride, int nrows,
                                             int slot0, bool fresh, float* scale_slot,
                                             uint8_t* dst) {
  if (nrows == 16)
    e2m1_v_tile<true>(GlobalRows{src, stride}, 16, 0, true, scale_slot, dst);
  else
    e2m1_v_tile<false>(GlobalRows{src, stride}, nrows, slot0, fresh, scale_slot, dst);
}

// Query heads [h0, h1) of the page's tokens.  A thread keeps one unit of one
// token, so its sines and cosines stay in registers over the heads.
template <int kD, bool IL, bool NORM>
__device__ __forceinline__ void queries(const RotaryArgs& a, const float2* cs, long long row0,
                                        int nrows, int rot16, int h0, int h1) {
  const int D = kD ? kD : a.app.d.head_dim_k, upr = D / 16, groups = kThreads / upr;
  const int g = threadIdx.x / upr, j = threadIdx.x - g * upr;
  // P * Dk <= 2048: a group of threads a token at least
  const int hs = groups / nrows, i = g / hs;
  if (g >= groups || i >= nrows) return;
  const UnitPlace p = unit_place(j, rot16, upr);
  float2 c[8];
  if (p.turn) unit_angles<IL, NORM>(cs + i * rot16 * 8, j, rot16, c);
  const UnitNorm norm = unit_norm<NORM>(a.q_norm, a.norm_eps, D, p);
  const uint16_t* q = a.q + (row0 + i) * a.q_stride;
  uint16_t* out = a.q_out + (row0 + i) * a.Hq * D;
  constexpr int kQ = kAhead;
  for (int h = h0 + g - i * hs; h < h1; h += kQ * hs) {
    uint4 r[kQ][2];
#pragma unroll
    for (int k = 0; k < kQ; ++k)
      if (h + k * hs < h1) {
        const uint4* src = reinterpret_cast<const uint4*>(q + (long long)(h + k * hs) * D);
        r[k][0] = __ldcs(src + p.c0);
        r[k][1] = __ldcs(src + p.c1);
      }
#pragma unroll
    for (int k = 0; k < kQ; ++k)
      if (h + k * hs < h1) {
        float x[16];
        unit_turn<IL, NORM>(r[k][0], r[k][1], p.turn, c, norm, x);
        uint4* o = reinterpret_cast<uint4*>(out + (long long)(h + k * hs) * D);
        o[p.c0] = pack8_bf16(x);
        o[p.c1] = pack8_bf16(x + 8);
      }
  }
}

// Two fp32 products or sums at a time
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}

// A unit's values of a head of 128 as packed pairs: x[j], x[4 + j] hold both values of the pairs
// 2j and 2j + 1 (first values in x[j], second in x[4 + j]).
template <bool IL>
__device__ __forceinline__ void unit_pairs(uint4 a, uint4 b, uint64_t (&x)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = IL ? w[2 * j] : w[j], v = IL ? w[2 * j + 1] : w[4 + j];
    x[j] = IL ? pack2(bf16_lo(u), bf16_lo(v)) : pack2(bf16_lo(u), bf16_hi(u));
    x[4 + j] = IL ? pack2(bf16_hi(u), bf16_hi(v)) : pack2(bf16_lo(v), bf16_hi(v));
  }
}

// The same for heads of 128 that are normalised: the weights and the sums take the registers
// that the loads in flight would, so a thread's come asynchronously through 32 bytes of shared
// memory each of its own.  The CTA's 32 groups of 8 threads sweep the tokens' heads in order.
// The fp32 arithmetic is packed, two values each.  (8 prompts of 1k-4k tokens: loads into registers
// 185 us, slots with a group a token 178, this with single products 172, packed 169; three CTAs an
// SM 179, queries and keys in kernels of their own 194, two CTAs a page 184.)
// angles(): works out the page's angles into cs, for the whole CTA; the first loads are on their
// way before it.
template <bool IL, class Angles>
__device__ __forceinline__ void queries_norm_128(const RotaryArgs& a, const float2* cs,
                                                 uint32_t at, long long row0, int nrows,
                                                 int rot16, int h0, int h1, const Angles& angles) {
  constexpr int kGroups = kThreads / 8;
  const int g = threadIdx.x >> 3, j = threadIdx.x & 7, nh = h1 - h0, items = nrows * nh;
  const UnitPlace p = unit_place(j, rot16, 8);
  const bool normed = a.q_norm != nullptr;
  uint64_t weight[8];
  if (normed)
    unit_pairs<IL>(reinterpret_cast<const uint4*>(a.q_norm)[p.c0],
                   reinterpret_cast<const uint4*>(a.q_norm)[p.c1], weight);
  const uint64_t minus = pack2(-1.0f, -1.0f);
  // (token, head) of an item, kGroups further at each step
  const int dt = kGroups / nh, dh = kGroups - dt * nh;
  auto next = [&](int& i, int& h) {
    i += dt;
    h += dh;
    if (h >= nh) {
      h -= nh;
      ++i;
    }
  };
  int fi = g / nh, fh = g - fi * nh;  // the next item to fetch
  auto fetch = [&](uint32_t slot) {
    if (fi < nrows) {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (row0 + fi) * a.q_stride + (h0 + fh) * 128);
      copy16(at + slot, src + p.c0);
      copy16(at + slot + kHalfSlot, src + p.c1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next(fi, fh);
  };
  int i = fi, h = fh;
#pragma unroll 1
  for (int k = 0; k < kDepth; ++k) fetch(k * kSlot);
  angles();
  uint32_t slot = 0;
  for (int m = g; m < items; m += kGroups) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    const uint4 r0 = take16(at + slot), r1 = take16(at + slot + kHalfSlot);
    fetch(slot);  // (this thread alone reads and fills its slots)
    uint64_t x[8];
    unit_pairs<IL>(r0, r1, x);
    if (normed) {
      uint64_t s0 = mul2(x[0], x[0]), s1 = mul2(x[4], x[4]);
#pragma unroll
      for (int k = 1; k < 4; ++k) {
        s0 = fma2(x[k], x[k], s0);
        s1 = fma2(x[4 + k], x[4 + k], s1);
      }
      const float2 u = unpack2(s0), v = unpack2(s1);
      float ss = (u.x + u.y) + (v.x + v.y);
      const uint32_t lanes = 0xFFu << (threadIdx.x & 24);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(lanes, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.0f / 128, a.norm_eps));
      const uint64_t rr = pack2(r, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = mul2(mul2(x[k], rr), weight[k]);
    }
    if (p.turn) {
      const float2* row = cs + i * rot16 * 8;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = IL ? (k < 2 ? 2 * j + k : 2 * (j + rot16) + k - 2) : 4 * j + k;
        const ulonglong2 t = reinterpret_cast<const ulonglong2*>(row)[angle_chunk<true>(c)];
        const uint64_t y = mul2(x[4 + k], mul2(t.y, minus)), z = mul2(x[k], t.y);
        x[k] = fma2(x[k], t.x, y);
        x[4 + k] = fma2(x[4 + k], t.x, z);
      }
    }
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 u = unpack2(x[k]), v = unpack2(x[4 + k]);
      w[IL ? 2 * k : k] = IL ? pack_bf16(u.x, v.x) : pack_bf16(u.x, u.y);
      w[IL ? 2 * k + 1 : 4 + k] = IL ? pack_bf16(u.y, v.y) : pack_bf16(v.x, v.y);
    }
    uint4* o = reinterpret_cast<uint4*>(a.q_out + ((row0 + i) * a.Hq + h0 + h) * 128);
    o[p.c0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[p.c1] = make_uint4(w[4], w[5], w[6], w[7]);
    next(i, h);
    slot = slot + kSlot == kDepth * kSlot ? 0 : slot + kSlot;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The part's kv heads of the page: a warp a tile.
template <int kD, bool IL, bool NORM, bool FP4>
__device__ __forceinline__ void keys_values(const RotaryArgs& a, const float2* cs, uint32_t slots, int r,
                                            long long jp, long long L0, long long row0, int nrows,
                                            int slot0, int rot16) {
  const AppendArgs& ap = a.app;
  const kv_pool_desc& d = ap.d;
  const int P = d.page_size, H = d.num_kv_heads, S = gridDim.y, part = blockIdx.y;
  const int warp = threadIdx.x >> 5;
  const int pg = ap.page_table[(long long)r * ap.max_pages + jp];
  if (pg < 0 || pg >= d.num_pages) {
    if (threadIdx.x == 0) set_error(d.ctl, KV_ERR_BAD_PAGE_ID);
    return;
  }
  const bool fresh = jp * P >= L0;  // popped by this call
  // a partly filled page that this call's pops handed to a later request is
  // not written through the stale mapping
  if (!fresh && d.tags[pg] != ap.exp_tags[(long long)r * ap.max_pages + jp]) return;
  const bool fp8 = d.dtype == KV_DTYPE_E4M3;
  const bool requant = fp8 && d.scale_mode == KV_SCALE_REQUANTIZE;
  const int es = fp8 ? 1 : 2, Dk = kD ? kD : d.head_dim_k, Dv = d.head_dim_v;
  const int h0 = (int)((long long)H * part / S), nh = (int)((long long)H * (part + 1) / S) - h0;
  uint8_t* kc = static_cast<uint8_t*>(d.k_cache);
  uint8_t* vc = static_cast<uint8_t*>(d.v_cache);
  for (int t = warp; t < 2 * nh; t += kWarps) {
    const int h = h0 + (t < nh ? t : t - nh);
    const long long ph = (long long)pg * H + h;
    if constexpr (FP4) {
      if (t < nh)
        key_tile_e2m1<IL, NORM>(ap.k_new + row0 * a.k_stride + (long long)h * 128, a.k_stride,
                                nrows, slot0, rot16, cs, a.k_norm, a.norm_eps, fresh,
                                d.k_scale + ph, kc + ph * kE2m1Tile);
      else
        value_tile_e2m1(ap.v_new + row0 * a.v_stride + (long long)h * 128, a.v_stride, nrows,
                        slot0, fresh, d.v_scale + ph, vc + ph * kE2m1Tile);
      continue;
    } else if (t < nh) {
      const uint16_t* src = ap.k_new + row0 * a.k_stride + (long long)h * Dk;
      float* scale = fp8 ? d.k_scale + ph : nullptr;
      uint8_t* dst = kc + ph * P * Dk * es;
      if (kD == 128 && nrows == 16 && P == 16 && !NORM)
        key_page_16x128<IL>(src, a.k_stride, rot16, cs, fp8, scale, dst);
      else if (kD == 128 && NORM && nrows == 16 && P == 16 && a.k_norm != nullptr)
        key_page_norm_16x128<IL>(src, a.k_stride, rot16, cs, slots, a.k_norm, a.norm_eps, fp8,
                                 scale, dst);
      else
        key_tile_any<IL, NORM>(src, a.k_stride, nrows, Dk, rot16, cs, a.k_norm, a.norm_eps, fp8,
                               fresh, requant, scale, dst, slot0);
    } else {
      const uint16_t* src = ap.v_new + row0 * a.v_stride + (long long)h * Dv;
      float* scale = fp8 ? d.v_scale + ph : nullptr;
      uint8_t* dst = vc + ph * P * Dv * es;
      if (nrows == 16 && P == 16 && Dv == 128)
        v_page_16x128(src, a.v_stride, fp8, scale, dst);
      else
        tile_warp_generic(src, a.v_stride, nrows, Dv, fp8, fresh, scale, dst, true, P, slot0,
                          nullptr, requant);
    }
  }
}

// the tables before the queries' slots, in bytes
__host__ __device__ constexpr int norm_ring_offset(int P, int half) {
  return (int)(sizeof(Freq) + sizeof(float2) * P) * half;
}

// kD: head_dim_k when it is known (0: any); IL: neighbouring pairs; NORM: heads are normalised; FP4: a
// 4-bit pool (kernels of their own: the calls of its tiles cost the others registers)
template <int kD, bool IL, bool NORM, bool FP4>
__global__ void __launch_bounds__(kThreads, 2) append_rotary_kernel(const RotaryArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const AppendArgs& ap = a.app;
  const kv_pool_desc& d = ap.d;
  const int P = d.page_size, half = a.rotary_dim / 2, rot16 = a.rotary_dim / 16;
  Freq* freq = reinterpret_cast<Freq*>(smem);               // [rot / 2]
  float2* cs = reinterpret_cast<float2*>(freq + half);      // [tokens of the page][rot / 2] (cos, sin)
  // ---- the tables, while the plan kernel runs: it has waited for what ran
  // before it, and does not write them
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double f = a.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
    const int ax = a.pair_axis[i];
    Freq e;
    e.turns = __double2ll_rn((f - rint(f)) * 0x1p64);
    e.axis = ax < a.num_axes ? ax : -1;
    e.skew = isfinite(f) ? 0.0f : __int_as_float(0x7FFFFFFF);
    freq[i] = e;
  }
  pdl_wait();
  pdl_trigger();
  // (the served requests' rows are in order; a refused one's may run backwards, and none of
  // its items may hide a served one's)
  const int stop = d.ctl[KV_CTL_APPEND_STOP];
  if (stop <= 0) return;  // nothing is served, and nothing written
  const int r = ragged_owner(ap.new_indptr, ap.B, stop, P, blockIdx.x);
  const long long i0 = ap.new_indptr[r], i1 = ap.new_indptr[r + 1], n = i1 - i0;
  if (n <= 0 || i0 < 0 || i1 > a.total_new) return;  // (the plan has refused it)
  const int local = blockIdx.x - ragged_first(i0, P, r);
  const long long Lnew = ap.seq_lens[r], L0 = Lnew - n;
  const long long jp = L0 / P + local;
  const long long lo = max(jp * P, L0), hi = min((jp + 1) * P, Lnew);
  if (local < 0 || lo >= hi) return;
  const int nrows = (int)(hi - lo), slot0 = (int)(lo - jp * P);
  const long long row0 = i0 + (lo - L0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  // ---- the angles of the page's tokens
  auto angles = [&]() {
    bool bad_axis = false;
    for (int t = warp; t < nrows; t += kWarps)
      for (int i = lane; i < half; i += 32) {
        const Freq f = freq[i];
        long long turns = 0;
        if (f.axis >= 0)
          turns = (long long)((unsigned long long)(long long)
                                  a.positions[(long long)f.axis * a.total_new + row0 + t] *
                              (unsigned long long)f.turns);
        else
          bad_axis = true;
        float2 v;
        sincospif(__ll2float_rn(turns) * 0x1p-63f + f.skew, &v.y, &v.x);
        if (NORM) {  // two pairs' cosines, then their sines: operands of the packed products
          float* at = reinterpret_cast<float*>(cs + t * half + 2 * angle_chunk<NORM>(i >> 1)) + (i & 1);
          at[0] = v.x;
          at[2] = v.y;
        } else {
          cs[t * half + i] = v;
        }
      }
    if (bad_axis) set_error(d.ctl, KV_ERR_INVALID_ARG);
    __syncthreads();
  };
  const int S = gridDim.y, part = blockIdx.y;
  // (NORM, heads of 128: this thread's slots)
  const uint32_t slots = smem_u32(smem) + norm_ring_offset(P, half) + 16 * threadIdx.x;
  const int h0 = (int)((long long)a.Hq * part / S), h1 = (int)((long long)a.Hq * (part + 1) / S);
  if (NORM && kD == 128 && h1 > h0) {
    queries_norm_128<IL>(a, cs, slots, row0, nrows, rot16, h0, h1, angles);
  } else {
    angles();
    if (a.q != nullptr) queries<kD, IL, NORM>(a, cs, row0, nrows, rot16, h0, h1);
  }
  keys_values<kD, IL, NORM, FP4>(a, cs, slots, r, jp, L0, row0, nrows, slot0, rot16);
}

}  // namespace

cudaError_t launch_append_rotary(const RotaryArgs& a, cudaStream_t s, int* launches) {
  cudaError_t e = launch_append_plan(a.app, s, launches);
  if (e != cudaSuccess || a.total_new == 0) return e;
  const int sms = sm_count();
  const int P = a.app.d.page_size;
  const long long items = ragged_items(a.total_new, a.app.B, P);
  // few pages: their heads are split, up to one wave of CTAs
  int split = (int)min(8LL, max(1LL, 2LL * sms / items));
  split = min(split, a.app.d.num_kv_heads);
  // at most 32 KB: P * Dk <= 2048
  size_t smem = (sizeof(Freq) + sizeof(float2) * (size_t)P) * (a.rotary_dim / 2);
  const bool il = a.interleaved != 0;
  const bool norm = a.q_norm != nullptr || a.k_norm != nullptr;
  const bool fp4 = a.app.d.dtype == KV_DTYPE_E2M1;
  // [4-bit, head_dim_k 128, any][neighbouring pairs][norm]
  static constexpr void (*const kKernels[3][2][2])(RotaryArgs) = {
      {{append_rotary_kernel<128, false, false, true>, append_rotary_kernel<128, false, true, true>},
       {append_rotary_kernel<128, true, false, true>, append_rotary_kernel<128, true, true, true>}},
      {{append_rotary_kernel<128, false, false, false>, append_rotary_kernel<128, false, true, false>},
       {append_rotary_kernel<128, true, false, false>, append_rotary_kernel<128, true, true, false>}},
      {{append_rotary_kernel<0, false, false, false>, append_rotary_kernel<0, false, true, false>},
       {append_rotary_kernel<0, true, false, false>, append_rotary_kernel<0, true, true, false>}}};
  const auto kernel = kKernels[fp4 ? 0 : a.app.d.head_dim_k == 128 ? 1 : 2][il][norm];
  if (norm && a.app.d.head_dim_k == 128) {
    smem = norm_ring_offset(P, a.rotary_dim / 2) + kDepth * 32 * kThreads;
    // (the largest page's: the same from every thread that may be between this and its launch)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)norm_ring_offset(16, 64) + kDepth * 32 * kThreads);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(kernel, dim3((unsigned)items, split), dim3(kThreads), smem, s, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
