// prefill.cu -- paged_prefill_attn: causal attention of many new tokens of a
// ragged batch over the paged cache.
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace kvfp8 {
namespace {

constexpr int kThreads = 256, kD = 128, kP = 16;

__device__ __forceinline__ int row_owner(const int32_t* indptr, int B, long long t) {
  int lo = 0, hi = B;  // the last r with indptr[r] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (indptr[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// One warp per (query token, head); lane l holds dims 4l .. 4l+3.
template <bool FP8>
__global__ void __launch_bounds__(kThreads) prefill_simple_kernel(const PrefillArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= (long long)a.total_q * a.Hq) return;
  const long long t = item / a.Hq;
  const int h = (int)(item % a.Hq), H = a.d.num_kv_heads, kvh = h / a.G;
  const int r = row_owner(a.q_indptr, a.B, t);
  const long long q0 = a.q_indptr[r], q1 = a.q_indptr[r + 1], L = a.seq_lens[r];
  if (t < q0 || t >= q1) return;
  if (a.abort_mask != nullptr && a.abort_mask[r] != 0) return;
  if (L < 0 || (L + kP - 1) / kP > a.max_pages || q0 < 0 || q1 > a.total_q) {
    if (lane == 0) set_error(a.d.ctl, KV_ERR_INVALID_ARG);
    return;
  }
  const long long seen = L - (q1 - q0) + (t - q0) + 1;  // visible positions
  const uint2 qw = *reinterpret_cast<const uint2*>(a.q + item * kD + 4 * lane);
  const float q[4] = {bf16_lo(qw.x), bf16_hi(qw.x), bf16_lo(qw.y), bf16_hi(qw.y)};
  float o[4] = {0, 0, 0, 0}, M = -INFINITY, l = 0.0f;
  for (long long j = 0; j * kP < seen; ++j) {
    const int p = a.page_table[(long long)r * a.max_pages + j];
    if (p < 0 || p >= a.d.num_pages) {
      if (lane == 0) set_error(a.d.ctl, KV_ERR_BAD_PAGE_ID);
      return;
    }
    const long long ph = (long long)p * H + kvh;
    const float ks = FP8 ? a.d.k_scale[ph] : 1.0f, vs = FP8 ? a.d.v_scale[ph] : 1.0f;
    const int nv = (int)min((long long)kP, seen - j * kP);
    float s[kP], mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      float k[4];
      if (FP8) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(
            static_cast<const uint8_t*>(a.d.k_cache) + (ph * kP + i) * kD + 4 * lane);
        const float2 x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(w & 0xFFFF, __NV_E4M3)));
        const float2 y = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(w >> 16, __NV_E4M3)));
        k[0] = x.x, k[1] = x.y, k[2] = y.x, k[3] = y.y;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(
            static_cast<const uint16_t*>(a.d.k_cache) + (ph * kP + i) * kD + 4 * lane);
        k[0] = bf16_lo(w.x), k[1] = bf16_hi(w.x), k[2] = bf16_lo(w.y), k[3] = bf16_hi(w.y);
      }
      const float dot = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]);
      s[i] = i < nv ? dot * ks * a.sm_scale_log2 : -INFINITY;
      mx = fmaxf(mx, s[i]);
    }
    const float Mn = fmaxf(M, mx), al = exp2f(M - Mn);
    l *= al;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= al;
    M = Mn;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      if (i >= nv) continue;
      const float pr = exp2f(s[i] - M);
      l += pr;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const long long at = (ph * kD + 4 * lane + e) * kP + i;
        const float v = FP8 ? __half2float(__half(__nv_cvt_fp8_to_halfraw(
                                  static_cast<const uint8_t*>(a.d.v_cache)[at], __NV_E4M3))) * vs
                            : bf16_bits_to_f32(static_cast<const uint16_t*>(a.d.v_cache)[at]);
        o[e] += pr * v;
      }
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const __nv_bfloat162 b0 = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
  const __nv_bfloat162 b1 = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
  *reinterpret_cast<uint2*>(a.out + item * kD + 4 * lane) = make_uint2(
      *reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
}

}  // namespace

size_t prefill_ws_bytes(const kv_pool_desc& d, int B, int Hq, int total_q) {
  (void)d, (void)B, (void)Hq, (void)total_q;
  return 256;
}

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t s, int* launches) {
  const long long items = (long long)a.total_q * a.Hq;
  const unsigned grid = (unsigned)((items + kThreads / 32 - 1) / (kThreads / 32));
  const cudaError_t e =
      a.d.dtype == KV_DTYPE_E4M3
          ? launch_pdl(prefill_simple_kernel<true>, dim3(grid), dim3(kThreads), 0, s, a)
          : launch_pdl(prefill_simple_kernel<false>, dim3(grid), dim3(kThreads), 0, s, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
