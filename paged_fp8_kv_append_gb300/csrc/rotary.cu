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
#include "append_tile.cuh"
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"
#include "ragged.cuh"

namespace kvfp8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAhead = 4;   // query units a thread has in flight

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

// (cos, sin) of a unit's 8 pairs from its token's row of them
template <bool IL>
__device__ __forceinline__ void unit_angles(const float2* row, int j, int rot16, float2 (&c)[8]) {
  const float4* a = reinterpret_cast<const float4*>(row + (IL ? 4 : 8) * j);
  const float4* b = IL ? reinterpret_cast<const float4*>(row + 4 * (j + rot16)) : a + 2;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 t = k < 2 ? a[k] : b[k - 2];
    c[2 * k] = make_float2(t.x, t.y);
    c[2 * k + 1] = make_float2(t.z, t.w);
  }
}

// The unit's values rotated: x[0..7] of chunk c0, x[8..15] of c1.
template <bool IL>
__device__ __forceinline__ void unit_turn(uint4 a, uint4 b, bool turn, const float2 (&c)[8],
                                          float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
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

// One (page, kv head) key tile by one warp: `nrows` rows from slot0 on; any
// shape, page and scale, a unit at a time (kept out of line: a fresh page's
// code stays small, and nothing of it lives across this call).
template <bool IL>
__device__ __noinline__ void key_tile_any(const uint16_t* src, long long stride, int nrows, int D,
                                          int rot16, const float2* cs, bool fp8, bool fresh,
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
    for (int u = lane; u < total; u += 32) {
      const int i = u / upr, j = u - i * upr;
      const UnitPlace p = unit_place(j, rot16, upr);
      const uint4* row = reinterpret_cast<const uint4*>(src + i * stride);
      float2 c[8];
      float x[16];
      if (p.turn) unit_angles<IL>(cs + i * rot16 * 8, j, rot16, c);
      unit_turn<IL>(row[p.c0], row[p.c1], p.turn, c, x);
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
  float x[4][16];
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 c[8];
    if (p.turn) unit_angles<IL>(cs + (i0 + 4 * k) * rot16 * 8, j, rot16, c);
    unit_turn<IL>(raw[k][0], raw[k][1], p.turn, c, x[k]);
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
    key_tile_any<IL>(src, stride, 16, 128, rot16, cs, true, true, false, scale_slot, dst, 0);
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

// Query heads [h0, h1) of the page's tokens.  A thread keeps one unit of one
// token, so its sines and cosines stay in registers over the heads.
template <int kD, bool IL>
__device__ __forceinline__ void queries(const RotaryArgs& a, const float2* cs, long long row0,
                                        int nrows, int rot16, int h0, int h1) {
  const int D = kD ? kD : a.app.d.head_dim_k, upr = D / 16, groups = kThreads / upr;
  const int g = threadIdx.x / upr, j = threadIdx.x - g * upr;
  // P * Dk <= 2048: a group of threads a token at least
  const int hs = groups / nrows, i = g / hs;
  if (g >= groups || i >= nrows) return;
  const UnitPlace p = unit_place(j, rot16, upr);
  float2 c[8];
  if (p.turn) unit_angles<IL>(cs + i * rot16 * 8, j, rot16, c);
  const uint16_t* q = a.q + (row0 + i) * a.q_stride;
  uint16_t* out = a.q_out + (row0 + i) * a.Hq * D;
  for (int h = h0 + g - i * hs; h < h1; h += kAhead * hs) {
    uint4 r[kAhead][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h + k * hs < h1) {
        const uint4* src = reinterpret_cast<const uint4*>(q + (long long)(h + k * hs) * D);
        r[k][0] = __ldcs(src + p.c0);
        r[k][1] = __ldcs(src + p.c1);
      }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h + k * hs < h1) {
        float x[16];
        unit_turn<IL>(r[k][0], r[k][1], p.turn, c, x);
        uint4* o = reinterpret_cast<uint4*>(out + (long long)(h + k * hs) * D);
        o[p.c0] = pack8_bf16(x);
        o[p.c1] = pack8_bf16(x + 8);
      }
  }
}

// The part's kv heads of the page: a warp a tile.
template <int kD, bool IL>
__device__ __forceinline__ void keys_values(const RotaryArgs& a, const float2* cs, int r,
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
    if (t < nh) {
      const uint16_t* src = ap.k_new + row0 * a.k_stride + (long long)h * Dk;
      float* scale = fp8 ? d.k_scale + ph : nullptr;
      uint8_t* dst = kc + ph * P * Dk * es;
      if (kD == 128 && nrows == 16 && P == 16)
        key_page_16x128<IL>(src, a.k_stride, rot16, cs, fp8, scale, dst);
      else
        key_tile_any<IL>(src, a.k_stride, nrows, Dk, rot16, cs, fp8, fresh, requant, scale, dst,
                         slot0);
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

// kD: head_dim_k when it is known (0: any); IL: neighbouring pairs
template <int kD, bool IL>
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
      cs[t * half + i] = v;
    }
  if (bad_axis) set_error(d.ctl, KV_ERR_INVALID_ARG);
  __syncthreads();
  const int S = gridDim.y, part = blockIdx.y;
  if (a.q != nullptr)
    queries<kD, IL>(a, cs, row0, nrows, rot16, (int)((long long)a.Hq * part / S),
                    (int)((long long)a.Hq * (part + 1) / S));
  keys_values<kD, IL>(a, cs, r, jp, L0, row0, nrows, slot0, rot16);
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
  const size_t smem = (sizeof(Freq) + sizeof(float2) * (size_t)P) * (a.rotary_dim / 2);
  const bool il = a.interleaved != 0;
  const auto kernel = a.app.d.head_dim_k == 128
                          ? (il ? append_rotary_kernel<128, true> : append_rotary_kernel<128, false>)
                          : (il ? append_rotary_kernel<0, true> : append_rotary_kernel<0, false>);
  e = launch_pdl(kernel, dim3((unsigned)items, split), dim3(kThreads), smem, s, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
