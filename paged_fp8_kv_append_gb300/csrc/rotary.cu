// rotary.cu -- kv_append_rotary: queries and keys rotated by their positions
// on one or several axes (a token's time, height and width), the keys and
// values quantised as they are written into the paged cache.
//
// Pair i of a head turns by a_i = position[axis(i)] * inv_freq[i]:
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a),
// the pair being dims (i, i + rot/2), or (2i, 2i + 1) when interleaved; dims
// from rot on pass through.  The product of a position and a frequency is
// taken in 64 bits and reduced to a fraction of a turn there, since a far
// position times a frequency near 1 keeps no fraction in fp32; sine and cosine
// of the fraction are fp32.  A rotated key stays in fp32 until its one
// rounding: to e4m3 by its page's scale (amax/448 of the page's rotated rows,
// as kv_append_quantize takes it of the rows it is given), or to bf16.
//
// Two launches: the append's plan kernel (append.cu: pages popped, tags
// stamped, lengths advanced), then this kernel, one CTA per (request, touched
// page): the angles of the page's tokens are computed once into shared memory
// and serve every query and key head of those tokens.
#include "append_tile.cuh"
#include "common.cuh"
#include "internal.h"
#include "quant.cuh"
#include "ragged.cuh"

namespace kvfp8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnits = 4;  // 16-value units of a key tile a lane holds (P * Dk <= 2048)

// Two 8-value chunks of a row hold 8 pairs: chunks j and j + rot/16 when the
// pairs lie rot/2 apart, chunks 2j and 2j + 1 when interleaved; units from
// rot/16 on pass through.
struct UnitPlace {
  int c0, c1;  // chunk numbers
  bool turn;
};
__device__ __forceinline__ UnitPlace unit_place(int j, int rot16, bool interleaved) {
  UnitPlace u;
  u.turn = j < rot16;
  const bool apart = u.turn && !interleaved;
  u.c0 = apart ? j : 2 * j;
  u.c1 = apart ? j + rot16 : 2 * j + 1;
  return u;
}

// The unit's 16 values rotated: x[0..7] from chunk c0, x[8..15] from c1; cs:
// (cos, sin) of its 8 pairs.
__device__ __forceinline__ void unit_turn(uint4 a, uint4 b, const UnitPlace& u, bool interleaved,
                                          const float2* cs, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
  }
  if (!u.turn) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 t = cs[k];
    float& p = interleaved ? x[2 * k] : x[k];
    float& q = interleaved ? x[2 * k + 1] : x[8 + k];
    const float p0 = p, q0 = q;
    p = p0 * t.x - q0 * t.y;
    q = q0 * t.x + p0 * t.y;
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

// 8 codes of x / s (the quotient to fp32 by one corrected product where the
// scale allows it, as the append kernels divide)
__device__ __forceinline__ uint2 codes8(const float* x, float s, float rs) {
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = e4m3x2(div_by_scale(x[2 * k], s, rs), div_by_scale(x[2 * k + 1], s, rs));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One (page, kv head) key tile by one warp: `nrows` rows from slot0 on.
__device__ void key_tile(const uint16_t* src, long long stride, int nrows, int D, int rot16,
                         bool interleaved, const float2* cs, bool fp8, bool fresh, bool requant,
                         float* scale_slot, uint8_t* dst, int slot0) {
  const int lane = threadIdx.x & 31, upr = D / 16, total = nrows * upr;
  float x[kUnits][16];
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int u = lane + 32 * k;
    if (u < total) {
      const int i = u / upr, j = u - i * upr;
      const UnitPlace p = unit_place(j, rot16, interleaved);
      const uint4* row = reinterpret_cast<const uint4*>(src + i * stride);
      unit_turn(row[p.c0], row[p.c1], p, interleaved, cs + (i * rot16 + j) * 8, x[k]);
#pragma unroll
      for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[k][e]));
    }
  }
  float s = 1.0f;
  if (fp8) {
    m = warp_max(m);
    if (fresh) {
      s = scale_from_amax(m);
      if (lane == 0) *scale_slot = s;
    } else {
      s = *scale_slot;
      const float s_new = scale_from_amax(m);
      if (requant && s_new > s) {  // a larger scale for the new rows: re-encode the old ones
        requant_block(dst, slot0, D, false, 0, s, s_new, lane, 32);
        __syncwarp();
        if (lane == 0) *scale_slot = s_new;
        s = s_new;
      }
    }
  }
  const float rs = __frcp_rn(s);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int u = lane + 32 * k;
    if (u < total) {
      const int i = u / upr, j = u - i * upr;
      const UnitPlace p = unit_place(j, rot16, interleaved);
      const long long at = (long long)(slot0 + i) * D;
      if (fp8) {
        *reinterpret_cast<uint2*>(dst + at + 8 * p.c0) = codes8(x[k], s, rs);
        *reinterpret_cast<uint2*>(dst + at + 8 * p.c1) = codes8(x[k] + 8, s, rs);
      } else {
        uint4* o = reinterpret_cast<uint4*>(dst + 2 * at);
        o[p.c0] = pack8_bf16(x[k]);
        o[p.c1] = pack8_bf16(x[k] + 8);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) append_rotary_kernel(const RotaryArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  float2* cs = reinterpret_cast<float2*>(smem);  // [tokens of the page][rot / 2] (cos, sin)
  pdl_wait();
  pdl_trigger();
  const AppendArgs& ap = a.app;
  const kv_pool_desc& d = ap.d;
  const int P = d.page_size;
  const int r = ragged_owner(ap.new_indptr, ap.B, P, blockIdx.x);
  if (r >= d.ctl[KV_CTL_APPEND_STOP]) return;  // not served: nothing of it is written
  const long long i0 = ap.new_indptr[r], i1 = ap.new_indptr[r + 1], n = i1 - i0;
  if (n <= 0) return;
  const int local = blockIdx.x - ragged_first(i0, P, r);
  if (i0 < 0 || i1 > a.total_new) {
    if (threadIdx.x == 0 && local == 0) set_error(d.ctl, KV_ERR_INVALID_ARG);
    return;
  }
  const long long Lnew = ap.seq_lens[r], L0 = Lnew - n;
  const long long jp = L0 / P + local;
  const long long lo = max(jp * P, L0), hi = min((jp + 1) * P, Lnew);
  if (local < 0 || lo >= hi) return;
  const int nrows = (int)(hi - lo), slot0 = (int)(lo - jp * P);
  const long long row0 = i0 + (lo - L0);
  // ---- the angles of the page's tokens
  const int half = a.rotary_dim / 2, rot16 = a.rotary_dim / 16;
  const bool il = a.interleaved != 0;
  bool bad_axis = false;
  for (int e = threadIdx.x; e < nrows * half; e += kThreads) {
    const int t = e / half, i = e - t * half, ax = a.pair_axis[i];
    double turn = 0.0;
    if (ax < a.num_axes) {
      const double angle = (double)a.positions[(long long)ax * a.total_new + row0 + t] * a.inv_freq[i];
      turn = angle * 0.15915494309189535;  // 1 / (2 pi)
      turn -= rint(turn);
    } else {
      bad_axis = true;
    }
    float2 v;
    sincospif((float)(2.0 * turn), &v.y, &v.x);
    cs[e] = v;
  }
  if (bad_axis) set_error(d.ctl, KV_ERR_INVALID_ARG);
  __syncthreads();
  // ---- queries
  const int Dk = d.head_dim_k, Dv = d.head_dim_v, H = d.num_kv_heads, upr = Dk / 16;
  if (a.q != nullptr) {
    const int per_row = a.Hq * upr, total = nrows * per_row;
    for (int u = threadIdx.x; u < total; u += kThreads) {
      const int i = u / per_row, hu = u - i * per_row, h = hu / upr, j = hu - h * upr;
      const UnitPlace p = unit_place(j, rot16, il);
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (row0 + i) * a.q_stride + (long long)h * Dk);
      float x[16];
      unit_turn(src[p.c0], src[p.c1], p, il, cs + (i * rot16 + j) * 8, x);
      uint4* o = reinterpret_cast<uint4*>(a.q_out + ((row0 + i) * a.Hq + h) * Dk);
      o[p.c0] = pack8_bf16(x);
      o[p.c1] = pack8_bf16(x + 8);
    }
  }
  // ---- keys and values
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
  const int es = fp8 ? 1 : 2, warp = threadIdx.x >> 5;
  uint8_t* kc = static_cast<uint8_t*>(d.k_cache);
  uint8_t* vc = static_cast<uint8_t*>(d.v_cache);
  for (int t = warp; t < 2 * H; t += kWarps) {
    const int h = t < H ? t : t - H;
    const long long ph = (long long)pg * H + h;
    if (t < H) {
      key_tile(ap.k_new + row0 * a.k_stride + (long long)h * Dk, a.k_stride, nrows, Dk, rot16, il,
               cs, fp8, fresh, requant, fp8 ? d.k_scale + ph : nullptr, kc + ph * P * Dk * es,
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

}  // namespace

cudaError_t launch_append_rotary(const RotaryArgs& a, cudaStream_t s, int* launches) {
  cudaError_t e = launch_append_plan(a.app, s, launches);
  if (e != cudaSuccess || a.total_new == 0) return e;
  const int P = a.app.d.page_size;
  const unsigned items = (unsigned)ragged_items(a.total_new, a.app.B, P);
  // at most 16 KB: P * Dk <= 2048
  const size_t smem = sizeof(float2) * (size_t)P * (a.rotary_dim / 2);
  e = launch_pdl(append_rotary_kernel, dim3(items), dim3(kThreads), smem, s, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
