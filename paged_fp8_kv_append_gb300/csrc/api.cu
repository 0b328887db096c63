// api.cu -- the C ABI declared in include/kvfp8.h: argument validation,
// launch configuration and workspace carve-up.  All compute is in the
// kernels of append.cu, rotary.cu, read.cu, verify.cu, release.cu, prefill.cu,
// decode_gqa.cu and decode_latent.cu; kv_decode_step chains them on one stream.
#include <math.h>

#include <new>

#include "internal.h"
#include "ragged.cuh"

using namespace kvfp8;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

namespace kvfp8 {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

kv_status decode_config(const kv_pool* pool, int B, int Hq, int T, DecodeConfig* cfg) {
  const kv_pool_desc& d = pool->d;
  if (B < 0 || Hq <= 0 || T <= 0) return KV_ERR_INVALID_ARG;
  if (d.layout == KV_LAYOUT_GQA) {
    if (Hq % d.num_kv_heads != 0) return KV_ERR_INVALID_ARG;
    const int G = Hq / d.num_kv_heads;
    // query rows per kv head, in blocks of 8 or 16 (one consumer warp each)
    const long long R = (long long)T * G;
    if (d.head_dim_k != 128 || d.head_dim_v != 128 || d.page_size != 16 || R > 64)
      return KV_ERR_UNSUPPORTED;
    // more than 8 rows: consumer warps of 16 rows, for 4-bit pools of 32 where the blocks of 16 are pairs and at most two of the eight warps serve
    // a (kv head, 32 rows) together (measured at the head of decode_e2m1.cu)
    const bool bf16 = d.dtype == KV_DTYPE_BF16, fp4 = d.dtype == KV_DTYPE_E2M1, wide = R > 8;
    const long long pairs = (R + 15) / 32, heads = d.num_kv_heads & -d.num_kv_heads;
    const bool wide32 = fp4 && wide && (R + 15) / 16 % 2 == 0 && pairs * heads >= 4;
    cfg->kind = fp4    ? (wide32 ? kGqaE2m1Rows32 : wide ? kGqaE2m1Rows16 : kGqaE2m1)
                : bf16 ? (wide ? kGqaBf16Wide : kGqaBf16)
                       : (wide ? kGqaE4m3Wide : kGqaE4m3);
    const int warp_rows = wide32 ? 32 : wide ? 16 : 8;
    const int warps = fp4 ? e2m1_split_warps(cfg->kind) : gqa_consumer_warps(cfg->kind);
    // heads per unit: the largest power of two <= 8 (<= 4 for bf16, whose
    // tiles are twice as large) dividing Hkv, with heads x row blocks dividing
    // the consumer warp count; 16-row blocks may be padded with whole unused
    // blocks until such a split exists; ring depth from the ring size
    int rbw = (int)((R + warp_rows - 1) / warp_rows);  // row blocks, one warp each
    int hs = 0;
    for (; rbw <= (wide ? 64 / warp_rows : 1); ++rbw) {
      hs = bf16 ? 4 : 8;
      while (hs > 0 && (d.num_kv_heads % hs != 0 || warps % (hs * rbw) != 0)) hs >>= 1;
      if (hs > 0) break;
    }
    if (hs == 0) return KV_ERR_UNSUPPORTED;  // no split of the consumers fits
    const int rb = rbw * warp_rows / 8;  // row blocks of 8 in the partial layout
    cfg->Hs = hs;
    cfg->stages = 0;
    if (!fp4) {  // (a warp of a 4-bit pool's kernel has a ring of its own)
      const int stage_bytes = 2 * hs * d.page_size * d.head_dim_k * (bf16 ? 2 : 1);
      cfg->stages = gqa_ring_bytes(cfg->kind) / stage_bytes;
      if (cfg->stages > gqa_max_stages()) cfg->stages = gqa_max_stages();
      // A consumer warp serves every (consumers/Hs)-th unit; the ring depth must
      // be a multiple of that stride so each warp sees every phase of the stages
      // it uses (parity waits cannot tell phase n from phase n-2).
      const int wph = warps / (hs * rbw);
      cfg->stages -= cfg->stages % wph;
      if (cfg->stages < 2 || cfg->stages < wph) return KV_ERR_UNSUPPORTED;
    }
    const int sms = sm_count();
    const int per_sm = sms <= 0 ? 0
                       : fp4    ? e2m1_split_ctas_per_sm(cfg->kind)
                                : gqa_split_ctas_per_sm(cfg->kind);
    if (sms <= 0 || per_sm <= 0) return KV_ERR_CUDA;
    cfg->grid = sms * per_sm;
    cfg->R8 = 8 * rb;
    cfg->HG = d.num_kv_heads / hs;
    cfg->unit_tokens = fp4 ? 2 * d.page_size : d.page_size;
    cfg->unit_extra = fp4 ? e2m1_unit_extra(cfg->kind) : 0;
    cfg->sub = fp4 ? warps / (hs * rbw) : 1;
    // the split kernel's CTAs plan a batch that fits their shared-memory
    // prefix cache themselves: no separate plan launch
    cfg->self_plan =
        ((fp4 || gqa_kind_self_plans(cfg->kind)) && B <= gqa_self_plan_max_batch()) ? 1 : 0;
    return KV_OK;
  }
  // latent layout: query rows (T tokens x Hq heads) in blocks of 64; the
  // row count stays far inside int range (2^20 rows)
  const int rb = latent_row_block();
  if ((long long)T * Hq > (1ll << 20)) return KV_ERR_UNSUPPORTED;
  if (d.head_dim_k != 576 || d.head_dim_v != 512 || d.page_size != 64 || (T * Hq) % rb != 0 ||
      d.dtype != KV_DTYPE_E4M3)
    return KV_ERR_UNSUPPORTED;
  const int sms = sm_count();
  const int per_sm = sms > 0 ? latent_split_ctas_per_sm() : 0;
  if (sms <= 0 || per_sm <= 0) return KV_ERR_CUDA;
  cfg->kind = kLatentE4m3;
  cfg->self_plan = 0;
  cfg->grid = sms * per_sm;
  cfg->R8 = rb;
  cfg->Hs = 1;
  cfg->HG = T * Hq / rb;
  cfg->stages = 0;
  cfg->unit_tokens = latent_unit_tokens();
  cfg->unit_extra = 0;
  cfg->sub = 1;
  return KV_OK;
}

size_t decode_ws_layout(const kv_pool_desc& d, int B, int Hkv, const DecodeConfig& cfg,
                        void* base, DecodeWs* ws) {
  // one partial slot per (CTA, segment) piece; segments are (request, head
  // group) or (request, row block); each slot holds Hs heads x R8 rows
  (void)Hkv;
  // (4-bit pools: cfg.sub of them)
  const long long slots = ((long long)B * cfg.HG + cfg.grid) * cfg.sub;
  size_t off = 0;
  const size_t o_pfx = off;
  off = align256(off + sizeof(int32_t) * (size_t)(B + 1));
  const size_t o_skip = off;
  off = align256(off + (size_t)B);
  const size_t o_ml = off;
  off = align256(off + sizeof(float) * 2 * (size_t)slots * cfg.Hs * cfg.R8);
  const size_t o_o = off;
  off = align256(off + sizeof(float) * (size_t)slots * cfg.Hs * cfg.R8 * d.head_dim_v);
  if (ws) {
    uint8_t* b = static_cast<uint8_t*>(base);
    ws->pfx = reinterpret_cast<int32_t*>(b + o_pfx);
    ws->rq_skip = b + o_skip;
    ws->ml_part = reinterpret_cast<float*>(b + o_ml);
    ws->o_part = reinterpret_cast<float*>(b + o_o);
    ws->bytes = off;
  }
  return off;
}

}  // namespace kvfp8

namespace {

kv_status decode_prepare(kv_pool* pool, int32_t B, int32_t Hq, int32_t T, const void* q,
                         const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                         const uint8_t* abort_mask, float sm_scale, void* out, void* workspace,
                         size_t workspace_bytes, bool need_inputs, bool need_out,
                         DecodeArgs* a, int* kind) {
  if (!pool) return KV_ERR_INVALID_ARG;
  const kv_pool_desc& d = pool->d;
  if (B < 0 || Hq <= 0 || T <= 0) return KV_ERR_INVALID_ARG;
  if (B > 0) {
    if (need_inputs && (!q || !page_table || !seq_lens || max_pages <= 0 || !aligned16(q) ||
                        !isfinite(sm_scale)))
      return KV_ERR_INVALID_ARG;
    // (every combine stores 8 bytes a lane)
    if (need_out && (!out || (reinterpret_cast<uintptr_t>(out) & 7u) != 0))
      return KV_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
      return KV_ERR_INVALID_ARG;
  }
  DecodeConfig cfg;
  const kv_status st = decode_config(pool, B, Hq, T, &cfg);
  if (st != KV_OK) return st;
  const int Hkv = d.num_kv_heads;
  DecodeArgs& x = *a;
  x.d = d;
  x.B = B;
  x.Hq = Hq;
  x.T = T;
  x.G = Hq / Hkv;
  x.R = (d.layout == KV_LAYOUT_GQA) ? T * x.G : T * Hq;
  x.q = static_cast<const uint16_t*>(q);
  x.page_table = page_table;
  x.max_pages = max_pages;
  x.seq_lens = seq_lens;
  x.abort_mask = abort_mask;
  x.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  x.out = static_cast<uint16_t*>(out);
  x.grid = cfg.grid;
  x.R8 = cfg.R8;
  x.Hs = cfg.Hs;
  x.HG = cfg.HG;
  x.stages = cfg.stages;
  x.unit_tokens = cfg.unit_tokens;
  x.unit_extra = cfg.unit_extra;
  x.sub = cfg.sub;
  x.self_plan = cfg.self_plan;
  x.exp_tags = nullptr;
  x.abort_out = nullptr;
  const size_t need = decode_ws_layout(d, B, Hkv, cfg, workspace, &x.ws);
  if (B > 0 && workspace_bytes < need) return KV_ERR_INVALID_ARG;
  *kind = cfg.kind;
  return KV_OK;
}

// Shapes that paged_prefill_attn takes.
kv_status prefill_check(const kv_pool_desc& d, int B, int Hq, int total_q) {
  if (B < 0 || Hq <= 0 || total_q < 0 || Hq % d.num_kv_heads != 0) return KV_ERR_INVALID_ARG;
  if (d.layout != KV_LAYOUT_GQA || d.head_dim_k != 128 || d.head_dim_v != 128 ||
      d.page_size != 16 || d.dtype == KV_DTYPE_E2M1)
    return KV_ERR_UNSUPPORTED;
  if (d.num_kv_heads > 4096) return KV_ERR_UNSUPPORTED;  // a page of all heads: 32-bit bytes
  // query rows of one kv head are counted in an int
  if ((long long)total_q * Hq > INT32_MAX) return KV_ERR_UNSUPPORTED;
  // so are items: 256 of those rows each, and one a request more
  if ((long long)total_q * (Hq / d.num_kv_heads) / 256 + B > INT32_MAX) return KV_ERR_UNSUPPORTED;
  return KV_OK;
}

// kv_append_rotary and kv_append_norm_rotary (norm weights may be NULL)
kv_status append_rotary(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                        int32_t total_new, const void* q, int64_t q_stride, const void* k_new,
                        int64_t k_stride, const void* v_new, int64_t v_stride,
                        const int32_t* new_indptr, int32_t max_new_per_req,
                        const int32_t* positions, int32_t num_axes, const uint8_t* pair_axis,
                        const double* inv_freq, int32_t rotary_dim, int32_t interleaved,
                        const void* q_norm, const void* k_norm, float norm_eps, void* q_out,
                        int32_t* page_table, uint32_t* exp_tags, int32_t max_pages_per_req,
                        int32_t* seq_lens) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  const kv_pool_desc& d = pool->d;
  if (B < 0 || total_new < 0 || max_new_per_req < 0 || max_pages_per_req <= 0 || num_q_heads < 0)
    return KV_ERR_INVALID_ARG;
  if (d.layout != KV_LAYOUT_GQA || !append_tile_fits(d)) return KV_ERR_UNSUPPORTED;
  if (num_axes < 1 || num_axes > 256 || rotary_dim <= 0 || rotary_dim % 16 != 0 ||
      rotary_dim > d.head_dim_k || (interleaved != 0 && interleaved != 1))
    return KV_ERR_INVALID_ARG;
  if (B == 0) return KV_OK;
  if (!new_indptr || !page_table || !exp_tags || !seq_lens) return KV_ERR_INVALID_ARG;
  if (total_new > 0) {
    const int64_t kw = (int64_t)d.num_kv_heads * d.head_dim_k;
    const int64_t vw = (int64_t)d.num_kv_heads * d.head_dim_v;
    const int64_t qw = (int64_t)num_q_heads * d.head_dim_k;
    if (!k_new || !v_new || !positions || !pair_axis || !inv_freq || !aligned16(k_new) ||
        !aligned16(v_new) || k_stride < kw || v_stride < vw || k_stride % 8 != 0 ||
        v_stride % 8 != 0)
      return KV_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out) || q_stride < qw ||
                            q_stride % 8 != 0))
      return KV_ERR_INVALID_ARG;
    // a block for each page that may be touched
    if (ragged_items(total_new, B, d.page_size) > INT32_MAX) return KV_ERR_UNSUPPORTED;
    // in place only row for row: at another stride a row's output is a later row's input
    if (num_q_heads > 0 && q_out == q && q_stride != qw && total_new > 1) return KV_ERR_INVALID_ARG;
  }
  RotaryArgs a = {};
  a.app.d = d;
  a.app.B = B;
  a.app.k_new = static_cast<const uint16_t*>(k_new);
  a.app.v_new = static_cast<const uint16_t*>(v_new);
  a.app.new_indptr = new_indptr;
  a.app.total_new = total_new;
  a.app.max_new = max_new_per_req < total_new ? max_new_per_req : total_new;
  a.app.page_table = page_table;
  a.app.exp_tags = exp_tags;
  a.app.max_pages = max_pages_per_req;
  a.app.seq_lens = seq_lens;
  a.q = num_q_heads > 0 ? static_cast<const uint16_t*>(q) : nullptr;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.Hq = num_q_heads;
  a.total_new = total_new;
  a.positions = positions;
  a.pair_axis = pair_axis;
  a.inv_freq = inv_freq;
  a.num_axes = num_axes;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved;
  a.q_norm = num_q_heads > 0 ? static_cast<const uint16_t*>(q_norm) : nullptr;
  a.k_norm = static_cast<const uint16_t*>(k_norm);
  a.norm_eps = norm_eps;
  int n = 0;
  const cudaError_t e = launch_append_rotary(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // namespace

extern "C" {

kv_status kv_pool_create(const kv_pool_desc* desc, kv_pool** out) {
  if (!desc || !out) return KV_ERR_INVALID_ARG;
  *out = nullptr;
  const kv_pool_desc& d = *desc;
  if (d.num_pages <= 0 || d.page_size <= 0 || d.page_size > 1024 || d.num_kv_heads <= 0 ||
      d.head_dim_k <= 0 || d.head_dim_v <= 0 || d.head_dim_k % 16 != 0 ||
      d.head_dim_v % 16 != 0 || d.head_dim_k > 1024 || d.head_dim_v > 1024)
    return KV_ERR_INVALID_ARG;
  if (d.dtype != KV_DTYPE_E4M3 && d.dtype != KV_DTYPE_BF16 && d.dtype != KV_DTYPE_E2M1)
    return KV_ERR_INVALID_ARG;
  if (d.layout != KV_LAYOUT_GQA && d.layout != KV_LAYOUT_LATENT) return KV_ERR_INVALID_ARG;
  if (d.scale_mode != KV_SCALE_FROZEN && d.scale_mode != KV_SCALE_REQUANTIZE)
    return KV_ERR_INVALID_ARG;
  if (!d.k_cache || !d.tags || !d.free_list || !d.ctl) return KV_ERR_INVALID_ARG;
  if (d.dtype == KV_DTYPE_E2M1) {
    // a tile's layout is that of the attention's fragments: one shape
    if (d.layout != KV_LAYOUT_GQA || d.page_size != 16 || d.head_dim_k != 128 ||
        d.head_dim_v != 128 || d.scale_mode != KV_SCALE_FROZEN || d.num_kv_heads > 4096)
      return KV_ERR_UNSUPPORTED;
    if (!d.k_scale || !d.v_scale) return KV_ERR_INVALID_ARG;
  }
  if (!aligned16(d.k_cache) || !aligned16(d.tags) || !aligned16(d.free_list) ||
      !aligned16(d.ctl))
    return KV_ERR_INVALID_ARG;
  if (d.layout == KV_LAYOUT_GQA) {
    if (!d.v_cache || !aligned16(d.v_cache)) return KV_ERR_INVALID_ARG;
    if (d.dtype == KV_DTYPE_E4M3 && (!d.k_scale || !d.v_scale)) return KV_ERR_INVALID_ARG;
    // the dim-major V tile of one page must fit the append kernel's staging
    if ((long long)d.head_dim_v * d.page_size * (d.dtype == KV_DTYPE_E4M3 ? 1 : 2) > 160 * 1024)
      return KV_ERR_UNSUPPORTED;
  } else {
    // a bf16 latent pool holds rows for appends and handoffs (attention over
    // it is not supported)
    if (d.num_kv_heads != 1 || d.head_dim_v > d.head_dim_k ||
        (d.dtype == KV_DTYPE_E4M3 && !d.k_scale))
      return KV_ERR_INVALID_ARG;
  }
  kv_pool* p = new (std::nothrow) kv_pool;
  if (!p) return KV_ERR_INVALID_ARG;
  p->d = d;
  p->last_launches = 0;
  *out = p;
  return KV_OK;
}

kv_status kv_pool_destroy(kv_pool* pool) {
  if (!pool) return KV_ERR_INVALID_ARG;
  delete pool;
  return KV_OK;
}

kv_status kv_append_quantize(kv_pool* pool, void* stream, int32_t B, const void* k_new,
                             const void* v_new, const int32_t* new_indptr,
                             int32_t max_new_per_req, int32_t* page_table, uint32_t* exp_tags,
                             int32_t max_pages_per_req, int32_t* seq_lens) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  const kv_pool_desc& d = pool->d;
  if (B < 0 || max_new_per_req < 0 || max_pages_per_req <= 0) return KV_ERR_INVALID_ARG;
  if (B == 0) return KV_OK;
  if (!new_indptr || !page_table || !exp_tags || !seq_lens) return KV_ERR_INVALID_ARG;
  if (max_new_per_req > 0) {
    if (!k_new || !aligned16(k_new)) return KV_ERR_INVALID_ARG;
    if (d.layout == KV_LAYOUT_GQA && (!v_new || !aligned16(v_new))) return KV_ERR_INVALID_ARG;
  }
  AppendArgs a;
  a.d = d;
  a.B = B;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.new_indptr = new_indptr;
  a.max_new = max_new_per_req;
  a.page_table = page_table;
  a.exp_tags = exp_tags;
  a.max_pages = max_pages_per_req;
  a.seq_lens = seq_lens;
  a.step_mask = nullptr;
  a.fuse_plan = false;
  a.from_pool = false;
  int n = 0;
  const cudaError_t e = launch_append(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kv_status kv_append_from_pool(kv_pool* pool, void* stream, int32_t B, const kv_pool* src,
                              const int32_t* src_page_table, int32_t src_max_pages_per_req,
                              const int32_t* src_seq_lens, int32_t* page_table,
                              uint32_t* exp_tags, int32_t max_pages_per_req, int32_t* seq_lens) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  if (!src || B < 0 || max_pages_per_req <= 0 || src_max_pages_per_req <= 0)
    return KV_ERR_INVALID_ARG;
  if (B == 0) return KV_OK;
  if (!src_page_table || !src_seq_lens || !page_table || !exp_tags || !seq_lens)
    return KV_ERR_INVALID_ARG;
  const kv_pool_desc& d = pool->d;
  const kv_pool_desc& sd = src->d;
  if (sd.dtype != KV_DTYPE_BF16 || sd.layout != d.layout || sd.num_kv_heads != d.num_kv_heads ||
      sd.head_dim_k != d.head_dim_k || sd.head_dim_v != d.head_dim_v ||
      sd.page_size != d.page_size)
    return KV_ERR_INVALID_ARG;
  if (!append_handoff_supported(d, B, src_max_pages_per_req)) return KV_ERR_UNSUPPORTED;
  AppendArgs a;
  a.d = d;
  a.B = B;
  a.k_new = nullptr;
  a.v_new = nullptr;
  a.new_indptr = nullptr;
  a.max_new = INT32_MAX;  // bounded by the page tables instead
  a.page_table = page_table;
  a.exp_tags = exp_tags;
  a.max_pages = max_pages_per_req;
  a.seq_lens = seq_lens;
  a.step_mask = nullptr;
  a.fuse_plan = false;
  a.from_pool = true;
  a.src = sd;
  a.src_page_table = src_page_table;
  a.src_max_pages = src_max_pages_per_req;
  a.src_lens = src_seq_lens;
  int n = 0;
  const cudaError_t e = launch_append(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kv_status kv_verify_tags(kv_pool* pool, void* stream, int32_t B, const int32_t* page_table,
                         const uint32_t* exp_tags, int32_t max_pages_per_req,
                         const int32_t* seq_lens, uint8_t* abort_mask) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  if (B < 0 || max_pages_per_req <= 0) return KV_ERR_INVALID_ARG;
  if (B == 0) return KV_OK;
  if (!page_table || !exp_tags || !seq_lens || !abort_mask) return KV_ERR_INVALID_ARG;
  VerifyArgs a;
  a.num_pages = pool->d.num_pages;
  a.page_size = pool->d.page_size;
  a.B = B;
  a.max_pages = max_pages_per_req;
  a.tags = pool->d.tags;
  a.page_table = page_table;
  a.exp_tags = exp_tags;
  a.seq_lens = seq_lens;
  a.abort_mask = abort_mask;
  int n = 0;
  const cudaError_t e = launch_verify(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

size_t kv_release_workspace_size(int32_t B) { return B < 0 ? 0 : release_ws_bytes(B); }

kv_status kv_release_pages(kv_pool* pool, void* stream, int32_t B, int32_t* page_table,
                           uint32_t* exp_tags, int32_t max_pages_per_req, int32_t* seq_lens,
                           const uint8_t* release_mask, void* workspace,
                           size_t workspace_bytes) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  if (B < 0 || max_pages_per_req <= 0) return KV_ERR_INVALID_ARG;
  if (B == 0) return KV_OK;
  if (!page_table || !exp_tags || !seq_lens || !workspace) return KV_ERR_INVALID_ARG;
  if (!aligned16(workspace) || workspace_bytes < release_ws_bytes(B)) return KV_ERR_INVALID_ARG;
  ReleaseArgs a;
  a.d = pool->d;
  a.B = B;
  a.max_pages = max_pages_per_req;
  a.page_table = page_table;
  a.exp_tags = exp_tags;
  a.seq_lens = seq_lens;
  a.mask = release_mask;
  a.mask_bits = 0xFF;
  a.offsets = static_cast<long long*>(workspace);
  int n = 0;
  const cudaError_t e = launch_release(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

size_t paged_decode_workspace_size(const kv_pool* pool, int32_t B, int32_t num_q_heads,
                                   int32_t q_tokens) {
  if (!pool || B < 0) return 0;
  DecodeConfig cfg;
  if (decode_config(pool, B, num_q_heads, q_tokens, &cfg) != KV_OK) return 0;
  return decode_ws_layout(pool->d, B, pool->d.num_kv_heads, cfg, nullptr, nullptr);
}

kv_status paged_decode_attn_split(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                                  int32_t q_tokens, const void* q, const int32_t* page_table,
                                  int32_t max_pages_per_req, const int32_t* seq_lens,
                                  const uint8_t* abort_mask, float sm_scale, void* workspace,
                                  size_t workspace_bytes) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  DecodeArgs a;
  int kind = 0;
  const kv_status st =
      decode_prepare(pool, B, num_q_heads, q_tokens, q, page_table, max_pages_per_req, seq_lens,
                     abort_mask, sm_scale, nullptr, workspace, workspace_bytes, true, false, &a,
                     &kind);
  if (st != KV_OK || B == 0) return st;
  int n = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = a.self_plan ? cudaSuccess : launch_decode_plan(a, s, &n);
  if (e == cudaSuccess) e = launch_decode_split(a, kind, s, &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kv_status paged_decode_attn_combine(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                                    int32_t q_tokens, const uint8_t* abort_mask, void* out,
                                    void* workspace, size_t workspace_bytes) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  DecodeArgs a;
  int kind = 0;
  const kv_status st =
      decode_prepare(pool, B, num_q_heads, q_tokens, nullptr, nullptr, 1, nullptr, abort_mask,
                     1.0f, out, workspace, workspace_bytes, false, true, &a, &kind);
  if (st != KV_OK || B == 0) return st;
  int n = 0;
  const cudaError_t e = launch_decode_combine(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kv_status paged_decode_attn(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                            int32_t q_tokens, const void* q, const int32_t* page_table,
                            int32_t max_pages_per_req, const int32_t* seq_lens,
                            const uint8_t* abort_mask, float sm_scale, void* out,
                            void* workspace, size_t workspace_bytes) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  if (B > 0 && !out) return KV_ERR_INVALID_ARG;
  // one argument set (and one validation) for the plan, the split and the combine
  DecodeArgs a;
  int kind = 0;
  const kv_status st =
      decode_prepare(pool, B, num_q_heads, q_tokens, q, page_table, max_pages_per_req, seq_lens,
                     abort_mask, sm_scale, out, workspace, workspace_bytes, true, true, &a, &kind);
  if (st != KV_OK || B == 0) return st;
  int n = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = a.self_plan ? cudaSuccess : launch_decode_plan(a, s, &n);
  if (e == cudaSuccess) e = launch_decode_split(a, kind, s, &n);
  if (e == cudaSuccess) e = launch_decode_combine(a, s, &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kv_status paged_decode_attn_checked(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                                    int32_t q_tokens, const void* q, const int32_t* page_table,
                                    const uint32_t* exp_tags, int32_t max_pages_per_req,
                                    const int32_t* seq_lens, float sm_scale, void* out,
                                    uint8_t* abort_mask, void* workspace,
                                    size_t workspace_bytes) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  if (B > 0 && (!out || !exp_tags || !abort_mask)) return KV_ERR_INVALID_ARG;
  DecodeArgs a;
  int kind = 0;
  const kv_status st =
      decode_prepare(pool, B, num_q_heads, q_tokens, q, page_table, max_pages_per_req, seq_lens,
                     nullptr, sm_scale, out, workspace, workspace_bytes, true, true, &a, &kind);
  if (st != KV_OK || B == 0) return st;
  a.exp_tags = exp_tags;
  a.abort_out = abort_mask;
  int n = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = a.self_plan ? cudaSuccess : launch_decode_plan(a, s, &n);
  if (e == cudaSuccess) e = launch_decode_split(a, kind, s, &n);
  if (e == cudaSuccess) e = launch_decode_combine(a, s, &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

size_t kv_decode_step_workspace_size(const kv_pool* pool, int32_t B, int32_t num_q_heads,
                                     int32_t q_tokens) {
  if (!pool || B < 0) return 0;
  DecodeConfig cfg;
  if (decode_config(pool, B, num_q_heads, q_tokens, &cfg) != KV_OK) return 0;
  const size_t dec = decode_ws_layout(pool->d, B, pool->d.num_kv_heads, cfg, nullptr, nullptr);
  return align256(dec) + release_ws_bytes(B);
}

kv_status kv_decode_step(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                         int32_t q_tokens, const uint8_t* leave_mask, const void* k_new,
                         const void* v_new, const int32_t* new_indptr, int32_t max_new_per_req,
                         int32_t* page_table, uint32_t* exp_tags, int32_t max_pages_per_req,
                         int32_t* seq_lens, const void* q, float sm_scale, void* out,
                         uint8_t* abort_mask, int32_t flags, void* workspace,
                         size_t workspace_bytes) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  const kv_pool_desc& d = pool->d;
  if (B < 0 || (flags & ~KV_STEP_REMOVE_ABORTED) != 0) return KV_ERR_INVALID_ARG;
  if (max_new_per_req < 0 || max_pages_per_req <= 0) return KV_ERR_INVALID_ARG;
  if (B == 0) return KV_OK;
  if (!new_indptr || !page_table || !exp_tags || !seq_lens || !abort_mask)
    return KV_ERR_INVALID_ARG;
  if (max_new_per_req > 0) {
    if (!k_new || !aligned16(k_new)) return KV_ERR_INVALID_ARG;
    if (d.layout == KV_LAYOUT_GQA && (!v_new || !aligned16(v_new))) return KV_ERR_INVALID_ARG;
  }
  // attention arguments and the workspace, before anything is launched
  DecodeArgs da;
  int kind = 0;
  kv_status st = decode_prepare(pool, B, num_q_heads, q_tokens, q, page_table, max_pages_per_req,
                                seq_lens, abort_mask, sm_scale, out, workspace, workspace_bytes,
                                true, true, &da, &kind);
  if (st != KV_OK) return st;
  const size_t need = kv_decode_step_workspace_size(pool, B, num_q_heads, q_tokens);
  if (need == 0 || workspace_bytes < need) return KV_ERR_INVALID_ARG;
  const size_t dec = need - release_ws_bytes(B);
  long long* rel_ws = reinterpret_cast<long long*>(static_cast<uint8_t*>(workspace) + dec);

  ReleaseArgs ra;
  ra.d = d;
  ra.B = B;
  ra.max_pages = max_pages_per_req;
  ra.page_table = page_table;
  ra.exp_tags = exp_tags;
  ra.seq_lens = seq_lens;
  ra.offsets = rel_ws;
  VerifyArgs va;
  va.num_pages = d.num_pages;
  va.page_size = d.page_size;
  va.B = B;
  va.max_pages = max_pages_per_req;
  va.tags = d.tags;
  va.page_table = page_table;
  va.exp_tags = exp_tags;
  va.seq_lens = seq_lens;
  va.abort_mask = abort_mask;
  AppendArgs aa;
  aa.d = d;
  aa.B = B;
  aa.k_new = static_cast<const uint16_t*>(k_new);
  aa.v_new = static_cast<const uint16_t*>(v_new);
  aa.new_indptr = new_indptr;
  aa.max_new = max_new_per_req;
  aa.page_table = page_table;
  aa.exp_tags = exp_tags;
  aa.max_pages = max_pages_per_req;
  aa.seq_lens = seq_lens;
  aa.step_mask = abort_mask;
  aa.from_pool = false;
  aa.fuse_plan = true;  // the append's plan kernel also writes the attention plan
  da.self_plan = 0;     // ... so the split kernel reads it
  aa.plan = da;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int n = 0;
  cudaError_t e = cudaSuccess;
  if (leave_mask != nullptr) {
    ra.mask = leave_mask;
    ra.mask_bits = 0xFF;
    e = launch_release(ra, s, &n);
  }
  if (e == cudaSuccess) e = launch_verify(va, s, &n);
  if (e == cudaSuccess) e = launch_append(aa, s, &n);
  if (e == cudaSuccess) e = launch_decode_split(da, kind, s, &n);
  if (e == cudaSuccess) e = launch_decode_combine(da, s, &n);
  if (e == cudaSuccess && (flags & KV_STEP_REMOVE_ABORTED) != 0) {
    ra.mask = abort_mask;
    ra.mask_bits = KV_ABORT_TAG;
    e = launch_release(ra, s, &n);
  }
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

kv_status kv_append_rotary(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                           int32_t total_new, const void* q, int64_t q_stride, const void* k_new,
                           int64_t k_stride, const void* v_new, int64_t v_stride,
                           const int32_t* new_indptr, int32_t max_new_per_req,
                           const int32_t* positions, int32_t num_axes, const uint8_t* pair_axis,
                           const double* inv_freq, int32_t rotary_dim, int32_t interleaved,
                           void* q_out, int32_t* page_table, uint32_t* exp_tags,
                           int32_t max_pages_per_req, int32_t* seq_lens) {
  return append_rotary(pool, stream, B, num_q_heads, total_new, q, q_stride, k_new, k_stride, v_new,
                       v_stride, new_indptr, max_new_per_req, positions, num_axes, pair_axis,
                       inv_freq, rotary_dim, interleaved, nullptr, nullptr, 0.0f, q_out, page_table,
                       exp_tags, max_pages_per_req, seq_lens);
}

kv_status kv_append_norm_rotary(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                                int32_t total_new, const void* q, int64_t q_stride,
                                const void* k_new, int64_t k_stride, const void* v_new,
                                int64_t v_stride, const int32_t* new_indptr,
                                int32_t max_new_per_req, const int32_t* positions,
                                int32_t num_axes, const uint8_t* pair_axis,
                                const double* inv_freq, int32_t rotary_dim, int32_t interleaved,
                                const void* q_norm, const void* k_norm, float norm_eps,
                                void* q_out, int32_t* page_table, uint32_t* exp_tags,
                                int32_t max_pages_per_req, int32_t* seq_lens) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  // a head's sum runs over a power of two of lanes, 16 dims each
  const int D = pool->d.head_dim_k;
  if ((q_norm || k_norm) && (D > 512 || (D & (D - 1)) != 0)) return KV_ERR_UNSUPPORTED;
  if (!(norm_eps >= 0.0f) || !isfinite(norm_eps) || !aligned16(q_norm) || !aligned16(k_norm))
    return KV_ERR_INVALID_ARG;
  return append_rotary(pool, stream, B, num_q_heads, total_new, q, q_stride, k_new, k_stride, v_new,
                       v_stride, new_indptr, max_new_per_req, positions, num_axes, pair_axis,
                       inv_freq, rotary_dim, interleaved, q_norm, k_norm, norm_eps, q_out,
                       page_table, exp_tags, max_pages_per_req, seq_lens);
}

kv_status kv_read_rows(kv_pool* pool, void* stream, int32_t B, const int32_t* page_table,
                       int32_t max_pages_per_req, const int32_t* seq_lens,
                       const int32_t* row_start, const int32_t* out_indptr, int32_t total_rows,
                       const uint8_t* abort_mask, void* k_out, void* v_out) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  if (B < 0 || total_rows < 0 || max_pages_per_req <= 0) return KV_ERR_INVALID_ARG;
  if (B == 0 || total_rows == 0) return KV_OK;
  if (!page_table || !seq_lens || !out_indptr || !k_out || !aligned16(k_out))
    return KV_ERR_INVALID_ARG;
  if (pool->d.layout == KV_LAYOUT_GQA && (!v_out || !aligned16(v_out))) return KV_ERR_INVALID_ARG;
  // a block for each page that may be touched
  if (ragged_items(total_rows, B, pool->d.page_size) > INT32_MAX) return KV_ERR_UNSUPPORTED;
  ReadArgs a;
  a.d = pool->d;
  a.B = B;
  a.max_pages = max_pages_per_req;
  a.total_rows = total_rows;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.row_start = row_start;
  a.out_indptr = out_indptr;
  a.abort_mask = abort_mask;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  int n = 0;
  const cudaError_t e = launch_read_rows(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

size_t paged_prefill_workspace_size(const kv_pool* pool, int32_t B, int32_t num_q_heads,
                                    int32_t total_q) {
  if (!pool || prefill_check(pool->d, B, num_q_heads, total_q) != KV_OK) return 0;
  return prefill_ws_bytes(pool->d, B, num_q_heads, total_q);
}

kv_status paged_prefill_attn(kv_pool* pool, void* stream, int32_t B, int32_t num_q_heads,
                             int32_t total_q, const void* q, const int32_t* q_indptr,
                             const int32_t* page_table, int32_t max_pages_per_req,
                             const int32_t* seq_lens, const uint8_t* abort_mask, float sm_scale,
                             void* out, void* workspace, size_t workspace_bytes) {
  if (!pool) return KV_ERR_INVALID_ARG;
  pool->last_launches = 0;
  const kv_status st = prefill_check(pool->d, B, num_q_heads, total_q);
  if (st != KV_OK) return st;
  if (B == 0 || total_q == 0) return KV_OK;
  if (!q || !q_indptr || !page_table || max_pages_per_req <= 0 || !seq_lens || !out ||
      !aligned16(q) || !aligned16(out) || !isfinite(sm_scale * 1.4426950408889634f) ||
      !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return KV_ERR_INVALID_ARG;
  const size_t need = prefill_ws_bytes(pool->d, B, num_q_heads, total_q);
  if (need == 0) return KV_ERR_CUDA;
  if (workspace_bytes < need) return KV_ERR_INVALID_ARG;
  PrefillArgs a;
  a.d = pool->d;
  a.B = B;
  a.Hq = num_q_heads;
  a.G = num_q_heads / pool->d.num_kv_heads;
  a.total_q = total_q;
  a.max_pages = max_pages_per_req;
  a.q = static_cast<const uint16_t*>(q);
  a.q_indptr = q_indptr;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.abort_mask = abort_mask;
  a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(out);
  a.workspace = workspace;
  int n = 0;
  const cudaError_t e = launch_prefill(a, static_cast<cudaStream_t>(stream), &n);
  pool->last_launches = n;
  return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

const char* kv_status_string(kv_status s) {
  switch (s) {
    case KV_OK: return "KV_OK";
    case KV_ERR_INVALID_ARG: return "KV_ERR_INVALID_ARG";
    case KV_ERR_UNSUPPORTED: return "KV_ERR_UNSUPPORTED";
    case KV_ERR_CUDA: return "KV_ERR_CUDA";
    case KV_ERR_OUT_OF_PAGES: return "KV_ERR_OUT_OF_PAGES";
    case KV_ERR_BAD_PAGE_ID: return "KV_ERR_BAD_PAGE_ID";
    case KV_ERR_TIMEOUT: return "KV_ERR_TIMEOUT";
    case KV_ERR_INTERNAL: return "KV_ERR_INTERNAL";
    case KV_ERR_TAG_MISMATCH: return "KV_ERR_TAG_MISMATCH";
  }
  return "KV_ERR_UNKNOWN";
}

int32_t kv_last_launch_count(const kv_pool* pool) { return pool ? pool->last_launches : 0; }

}  // extern "C"

namespace kvfp8 {

cudaError_t launch_decode_split(const DecodeArgs& a, int kind, cudaStream_t s, int* launches) {
  if (kind == kLatentE4m3) return launch_latent_split(a, s, launches);
  if (kind >= kGqaE2m1) return launch_e2m1_split(a, kind, s, launches);
  return launch_gqa_split(a, kind, s, launches);
}

}  // namespace kvfp8
