// prefill.cu -- paged_prefill_attn: causal attention of many new tokens of a
// ragged batch over the paged cache, on the tcgen05 tensor cores.
//
// "Smaller, faster, safer: running Kimi and GLM at scale", section
// "Quantizing the KV cache": attention reads the e4m3 cache and converts
// values as it reads them; bf16 is the baseline format.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j), j <= L - n + i,
// in one pass over the keys with a running reference and sum of each row.  What a row does not
// see does not reach it, whatever it is: scores are masked, pages' scales that are no numbers
// are kept beside the arithmetic, values that are not finite left out (find_hidden).
//
// Work decomposition.  A request's query rows of one kv head are row = t * G + g
// (token, head of the group); 256 of them are an item's two tiles of 128 rows
// (A and B).  A block is 128 tokens (8 pages), a unit half of one.  An item with at
// most 128 rows has one tile, and then A and B are the same rows over the two halves of
// each block, merged when the item ends.  Items are laid out request-major on an axis of
// costs, and the whole batch is cut into equal ranges, one per persistent CTA: every CTA
// works equally long whatever the lengths.  A CTA writes an item that lies wholly in its
// range; an item cut by a range's end leaves fp32 partials (o, reference, sum) for the
// combine kernel, at most two a CTA.
//
// Per CTA (one per SM, 15 warps of 128 registers):
//   softmax A (0-3), B (4-7)  a thread per row: a unit's 64 scores from tensor memory
//                   into registers, exp2 against the row's reference M as it stands, P back
//                   to tensor memory as the A operand of PV (e4m3 pools: f16; bf16 pools: two
//                   bf16 parts, which keep 16 bits of a weight as the decode attention does, for
//                   a second PV: one part took 854 us for four ragged prompts, two take 1,038, and
//                   a weight of 8 bits is off by 2^-9).  The unit's maximum is taken
//                   only in a first unit, for a row that has seen nothing yet, or when the
//                   P of a row sum to 2^15 or more (f16 P stay finite below that); M then
//                   grows if it must and the output accumulator is rescaled by the same
//                   warp.  Between two items the next item's query rows (f16 by an exact
//                   power of two a row, or bf16) go into shared memory, then the output
//   converters (8-11)  two warps for the keys, two for the values: global pages ->
//                   registers -> 128B-swizzled K-major tiles in shared memory, K
//                   [token][dim] and V [dim][token] (pages hold V dim-major: no
//                   transpose).  e4m3 codes become f16 exactly, bf16 is copied
//   MMA A (12), B (13)  S = Q K^T (M 128, N 64) a unit ahead of O += P V (M = N = 128),
//                   so that a tile's softmax finds its next scores when it has stored P
//   scheduler (14)  the CTA's pieces, one after the other into a ring that the other
//                   warps read, their query rows pulled into L2, the values that some of
//                   their rows must not see looked through
// Every wait is bounded (KV_ERR_TIMEOUT); tensor memory is freed on every path.
//
// What bounds it, and what was measured (64 query and 8 kv heads, e4m3, TFLOP/s of 4 Hq D
// a visible pair, of 1,943 that cuBLAS reaches in bf16):
//   2 x 2048 tokens behind 30k cached   3.20 ms, 1.33e15/s (68%): the tensor pipe is 68%
//     busy.  S of 64 columns reads its 32 KB of queries from shared memory again for each
//     unit (48 KB in 384 cycles where its products take 256); scores of 128 columns at a
//     time cost less there but leave no room in tensor memory to be a step ahead: 4.25 ms,
//     the softmax warps wait for their scores.
//   one prompt of 8192    0.94 ms, 1.16e15 (60%): the same, and about 8 us an item (6 of
//     them queries in) that the other items of the CTA hide in part.
//   16 tokens of 32 requests, 4k-32k cached   0.289 ms, 0.89e15, 3.6 TB/s of cache: 128 rows
//     make half the products of a block whose keys and values are the same 32 KB.  Bound
//     by the converters, a block in 2,600 cycles.
//   four ragged bf16 prompts, 96 heads   1.05 ms, 0.84e15 (43%): the tensor pipe is 72% busy,
//     0.29 of that with the weights' second parts.
// Two converter warps for each of K and V against four for both in turn: drafts 378 -> 292
// us, four ragged bf16 prompts 1,139 -> 965: a block's waits, page ids, fence and arrival
// are paid once for it, and keys do not wait for values (weights of one part then).  Eight
// converter warps leave 96 registers a thread, and the softmax then spills: chunk 3.3 -> 4.0 ms.  Pages by bulk copies
// or cp.async through 32 KB of shared memory were slower than the loads (a bulk copy is about
// 66 cycles of its warp, 16 a block).  All of the loops together have to stay small: the code
// is 90 KB (bf16: 84), a fifth of it seldom run, and variants that unrolled more ran slower by
// what the instruction cache misses (16 KB more in the loops: drafts 284 -> 335 us).
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"
#include "tcgen05.cuh"

namespace kvfp8 {
namespace {

constexpr int kD = 128, kP = 16;
constexpr int kTile = 128, kItemRows = 2 * kTile;  // query rows
constexpr int kBlk = 128, kBlkPages = kBlk / kP;   // tokens / pages of a key block
constexpr int kUnit = kBlk / 2, kUnitPages = kUnit / kP;
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kMmaWarp = kSoftWarps + kConvWarps;  // the scheduler is behind it
constexpr int kRing = 4;  // pieces in flight from the scheduler
constexpr int kThreads = (kMmaWarp + 3) * 32;
// Costs, about 0.65 us each (e4m3): a block of an item with two tiles, one of an item with a
// single tile (1.95 and 1.4 us: the keys and values are as many, the rows half), and what an
// item costs beside its blocks (queries in, output out).  At 2 : 1 for the blocks four ragged
// prompts take 922 us (bf16 1,092), at 3 : 2 871 (1,062), at 4 : 3 882 (1,062).  An item of two
// tiles, about 8 us, counts fewer of a bf16 pool's blocks, which take longer.  Measured on four shapes for both types (one prompt of
// 8k tokens and 64 heads, four ragged ones and 96, six and 32, one of 4k and 32; us):
//   e4m3, lead 10   1090 951 387 185        bf16, lead 10   1211 1056 396 197
//              11   1036 929 376 177                   11   1211 1056 398 193
//              12    997 907 371 172                   12   1218 1060 401 193
//              14    945 871 359 165                   14   1217 1063 405 194
//              16    951 872 360 163                   16   1219 1084 415 194
constexpr int kCostTwo = 3, kCostOne = 2;
__host__ __device__ inline int item_lead(int nrows, bool fp8) {
  return nrows > 128 ? (fp8 ? 14 : 11) : 9;
}
constexpr int kMeta = 4;  // block records in flight
// Where a unit's maximum is taken, the reference of a row of an e4m3 pool goes this far (binades)
// below it: f16 weights lose bits below 2^-14 and end at 2^-25, so what lies far below a row's
// largest keeps as many more; upwards 2^15 are allowed anyway.
constexpr float kRoom = 6.0f;

// shared memory: operand tiles of two 64-wide halves, [128 rows][128 B] each
constexpr int kHalf = 128 * 128, kTileBytes = 2 * kHalf;
constexpr int OFF_Q = 0;                          // tiles A, B
constexpr int OFF_K = OFF_Q + 2 * kTileBytes;     // 2 blocks
constexpr int OFF_V = OFF_K + 2 * kTileBytes;     // 2 blocks
constexpr int OFF_META = OFF_V + 2 * kTileBytes;  // [kMeta][8] float4
constexpr int OFF_MLB = OFF_META + kMeta * kBlkPages * 16;   // [128] float2
constexpr int OFF_HB = OFF_MLB + kTile * 8;                  // [128] float
constexpr int OFF_RING = OFF_HB + kTile * 4;                 // [kRing] Piece
constexpr int OFF_SPOIL = OFF_RING + kRing * 48;             // [kRing][128] uint8_t
constexpr int OFF_BAR = OFF_SPOIL + kRing * kD;
constexpr int kBars = 8 + 2 + 8 + 6 + 3 + 3 * kRing;
constexpr int OFF_MISC = OFF_BAR + kBars * 8;
constexpr int kSmem = OFF_MISC + 8;
// (with the 1 KB that a CTA has besides; one step more leaves 32 KB less of L1: drafts +7%)
static_assert(kSmem <= (196 - 1) * 1024, "shared memory budget");

// tensor memory columns: two S of 64 (P in the first half of each; bf16 pools: its second parts
// in the second) and O of each tile
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t tmem_o(int x) { return 256u + 128u * x; }

// kind::f16 instruction descriptor: M 128, f32 accumulate, both operands K-major
constexpr uint32_t idesc(bool bf16, uint32_t n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// flags of a key block, kept beside its scales
constexpr uint32_t kBadPage = 1, kWide = 2;  // an id out of range; V scales far from 1
// a page whose scales are no numbers (negative, infinite, NaN), and the same of that page alone
constexpr uint32_t kOdd = 4, kOddPage = 8;

// ------------------------------------------------------------------ plan

struct Ws {
  long long* pfx;   // [V+1] cost of the items before, per kv head
  int4* items;      // [V] {request, first row, rows, blocks}
  int4* cut;        // [grid] {item (-1: none), kv head, last CTA, 0}: the cut item a CTA begins
  float2* ml;       // [2 grid][256] (running max, sum; -1: a page that must not be read)
  float4* o;        // [2 grid][32][256]: 4 dims of a row
  size_t bytes;
};

__host__ __device__ inline long long item_first(long long q0, int G, int r) {
  return q0 * G / kItemRows + r;
}

long long item_count(int B, int G, int total_q) {
  return (long long)total_q * G / kItemRows + B;
}

Ws ws_layout(void* base, int B, int G, int total_q, int grid) {
  const size_t V = (size_t)item_count(B, G, total_q);
  size_t off = 0;
  uint8_t* b = static_cast<uint8_t*>(base);
  auto take = [&](size_t n) {
    uint8_t* p = b + off;
    off = (off + n + 255) & ~size_t(255);
    return p;
  };
  Ws w;
  w.pfx = reinterpret_cast<long long*>(take(8 * (V + 1)));
  w.items = reinterpret_cast<int4*>(take(16 * V));
  w.cut = reinterpret_cast<int4*>(take(16 * (size_t)grid));
  w.ml = reinterpret_cast<float2*>(take(8ull * 2 * grid * kItemRows));
  w.o = reinterpret_cast<float4*>(take(4ull * 2 * grid * kItemRows * kD));
  w.bytes = off;
  return w;
}

struct Args {
  PrefillArgs p;
  Ws ws;
  int V, grid;
};

constexpr int kPlanThreads = 1024;

// Whether request r (rows q0 .. q1-1) can be attended: its rows lie in q, and it has a length
// that its page table holds (positions of a block are ints).
__device__ __forceinline__ bool request_fits(const PrefillArgs& p, long long q0, long long q1,
                                             long long L) {
  return q0 <= q1 && q0 >= 0 && q1 <= p.total_q && L >= 0 && (L + kP - 1) / kP <= p.max_pages &&
         L <= INT_MAX - 2 * kBlk;
}

// One CTA: every item's request, rows and blocks, and the cost prefix.  Requests are checked by
// themselves, as a refused one's rows may lie behind every item or in another's; items are those
// of the requests before the first whose rows run backwards, so that their search is one of an
// increasing sequence.
__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const Args a) {
  pdl_wait();
  pdl_trigger();
  __shared__ long long sums[32];
  const PrefillArgs& p = a.p;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int first_back = p.B;  // the first of this thread's requests whose rows run backwards
  for (int r = threadIdx.x; r < p.B; r += kPlanThreads) {
    const long long q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1];
    const bool aborted = p.abort_mask != nullptr && p.abort_mask[r] != 0;
    if (q1 < q0) first_back = min(first_back, r);
    if (q1 < q0 || (!aborted && q0 != q1 && !request_fits(p, q0, q1, p.seq_lens[r])))
      set_error(p.d.ctl, KV_ERR_INVALID_ARG);
  }
  int served = p.B;
  if (__syncthreads_or(first_back < p.B)) {
    __shared__ int s_served;
    if (threadIdx.x == 0) s_served = p.B;
    __syncthreads();
    atomicMin(&s_served, first_back);
    __syncthreads();
    served = s_served;
  }
  long long carry = 0;
  for (int base = 0; base < a.V; base += kPlanThreads) {
    const int v = base + threadIdx.x;
    long long cost = 0;
    if (v < a.V) {
      int lo = 0, hi = served;  // the last r whose items begin at or before v
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (item_first(p.q_indptr[mid], p.G, mid) <= v) lo = mid; else hi = mid;
      }
      const int r = lo;
      const long long q0 = p.q_indptr[r], q1 = p.q_indptr[r + 1], n = q1 - q0;
      const long long L = p.seq_lens[r], row0 = (v - item_first(q0, p.G, r)) * kItemRows;
      int4 it = make_int4(r, 0, 0, 0);
      const bool aborted = p.abort_mask != nullptr && p.abort_mask[r] != 0;
      if (r < served && !aborted && request_fits(p, q0, q1, L) && row0 >= 0 && row0 < n * p.G) {
        it.y = (int)row0;
        it.z = (int)min((long long)kItemRows, n * p.G - row0);
        const long long seen = L - n + (row0 + it.z - 1) / p.G + 1;  // by the last row
        it.w = (int)max(1LL, (seen + kBlk - 1) / kBlk);
        cost = item_lead(it.z, p.d.dtype == KV_DTYPE_E4M3) +
               (long long)it.w * (it.z > kTile ? kCostTwo : kCostOne);
      }
      a.ws.items[v] = it;
    }
    long long s = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    if (lane == 31) sums[wid] = s;
    __syncthreads();
    if (wid == 0) {
      long long t = sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += x;
      }
      sums[lane] = t;
    }
    __syncthreads();
    if (v < a.V) a.ws.pfx[v] = carry + s - cost + (wid > 0 ? sums[wid - 1] : 0);
    carry += sums[31];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.ws.pfx[a.V] = carry;
}

// -------------------------------------------------------- a CTA's pieces

// The piece of an item (request r, kv head h, query rows row0 ..) that lies in a
// CTA's range of the cost axis: blocks b_lo .. b_hi-1 of the item's nb.
struct Piece {
  int r, h, row0, nrows;
  int b_lo, b_hi, nb, L;
  int n, q0, valid, apart;  // (apart: see find_hidden)
  __device__ __forceinline__ int seen_all(int G) const {  // tokens that every row sees
    return L - n + row0 / G + 1;
  }
  __device__ __forceinline__ bool both() const { return nrows > kTile; }
  __device__ __forceinline__ int w() const { return both() ? kCostTwo : kCostOne; }
  __device__ __forceinline__ int count() const { return b_hi - b_lo; }
};
static_assert(sizeof(Piece) == 48, "ring slots");

// The scheduler's place on the cost axis.
struct Walk {
  int v, h, lead;
  long long x0;  // cost position of (item v, head h)
  Piece s;
  // of its first block, and behind its last
  __device__ __forceinline__ long long blocks0() const { return x0 + lead; }
  __device__ __forceinline__ long long cost() const {
    return lead + (long long)s.nb * s.w();
  }
};

__device__ __forceinline__ int block_at(long long x, const Walk& c) {  // first block at or behind x
  const long long d = x - c.blocks0();
  if (d <= 0) return 0;
  return (int)min((long long)c.s.nb,
                  c.s.both() ? (d + kCostTwo - 1) / kCostTwo : (d + kCostOne - 1) / kCostOne);
}

__device__ __forceinline__ void walk_item(Walk& c, const Args& a) {
  const int4 it = a.ws.items[c.v];
  c.s.r = it.x;
  c.s.row0 = it.y;
  c.s.nrows = it.z;
  c.lead = item_lead(it.z, a.p.d.dtype == KV_DTYPE_E4M3);
  c.s.nb = it.w;
  c.s.L = a.p.seq_lens[it.x];
  c.s.q0 = a.p.q_indptr[it.x];
  c.s.n = a.p.q_indptr[it.x + 1] - c.s.q0;
}

__device__ __forceinline__ void walk_head(Walk& c, const Args& a, long long x_begin,
                                          long long x_end) {
  c.x0 = a.ws.pfx[c.v] * a.p.d.num_kv_heads + (long long)c.h * c.cost();
  c.s.h = c.h;
  c.s.b_lo = block_at(x_begin, c);
  c.s.b_hi = block_at(x_end, c);
  c.s.valid = 1;
}

// --------------------------------------------------------------- helpers

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <bool FP8>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  if (FP8) return pack_f16(lo, hi);
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]));
}
// 64 columns of this warp's lanes
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
// 16 columns times f, in place
__device__ __forceinline__ void tmem_scale16(uint32_t taddr, float f) {
  float r[16];
  tmem_ld16(taddr, r);
  uint32_t w[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(r[k] * f);
  tmem_st16u(taddr, w);
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Wait for phase `parity` of `bar`: false once a wait of the CTA has run out
// (kWaitLimitNs), which *abort_flag tells the others and the kernel's end reports.
// What follows a first probe (which itself waits a while) is out of line: the
// kernel's loops have to stay small in the instruction cache.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                     int info) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 15u) != 15u) continue;
    const uint64_t now = global_ns();
    if (t0 == 0) t0 = now;
    if (*abort_flag != 0 || now - t0 > kWaitLimitNs) {
      if (*abort_flag == 0) *abort_flag = info + 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity,
                                           volatile int* abort_flag, int info) {
  bool ok = mbar_try_wait(bar, parity & 1u);
  if (!ok) ok = wait_on(bar, parity & 1u, abort_flag, info);
  return __all_sync(0xffffffffu, ok);
}

// The K steps of one product in one piece of code, so that the predicates are set once
// and descriptors differ by constants (16-byte units; the second 64-wide half of a tile
// begins kHalf bytes behind the first).  ss4 / ts4: four steps of a half, the first
// accumulating iff `add`.
__device__ __forceinline__ void mma_ss4(uint32_t leader, uint32_t d, uint64_t a, uint64_t b,
                                        uint32_t id, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 a, b;\n"
      " setp.ne.b32 q, %5, 0;\n setp.ne.b32 p, %4, 0;\n setp.eq.u32 t, 0, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(add), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts4(uint32_t leader, uint32_t d, uint32_t a, uint64_t b,
                                        uint32_t id, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 b;\n .reg .b32 a;\n"
      " setp.ne.b32 q, %5, 0;\n setp.ne.b32 p, %4, 0;\n setp.eq.u32 t, 0, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " add.s32 a, %1, 8;\n add.s64 b, %2, 2;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 16;\n add.s64 b, %2, 4;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 24;\n add.s64 b, %2, 6;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(add), "r"(leader)
      : "memory");
}

// ---------------------------------------------- values that are not finite
//
// A weight of 0 times a value that is not finite is NaN: such a value of a token that not all of
// an item's rows see would reach those that do not.  The few such tokens of a piece (256 rows / G,
// and what its last block holds behind them) are looked through by the scheduler; if one has such
// a value, the piece's values are brought in by a loop of its own that zeroes it, and the output's
// end makes the dim NaN for the rows that see it.  (Blocks of tokens that every row sees need
// none of this: their NaN are the rows' own.)

// the request's j-th page, or page 0 where there is none
__device__ __forceinline__ long long page_or_0(const PrefillArgs& p, const Piece& pc, int j) {
  const int pg = j * kP < pc.L ? p.page_table[(long long)pc.r * p.max_pages + j] : 0;
  return pg >= 0 && pg < p.d.num_pages ? pg : 0;
}

// Whether one of the tokens from seen_all() to the piece's last block's end is not finite; sp[dim]
// = the first such token of the dim, counted from seen_all() (255: none that a row sees).  One
// warp.  (Out of line, or with twice as many pages in flight, the code grows and prompts lose
// 2-5%.)
template <bool FP8>
__device__ __forceinline__ bool find_hidden(const PrefillArgs& p, const Piece& pc, uint8_t* sp) {
  constexpr int kEs = FP8 ? 1 : 2, kQ = kEs, kAhead = 2 / kEs;  // 16-byte pieces of a dim; pages
  constexpr uint32_t kOnes = FP8 ? 0x7F7F7F7Fu : 0x7F807F80u;   // what a value not finite has
  constexpr uint32_t kLow = FP8 ? 0x01010101u : 0x00800080u;    // carries it into the sign
  constexpr uint32_t kSign = FP8 ? 0x80808080u : 0x80008000u;
  const int lane = threadIdx.x & 31;
  const int t0 = pc.seen_all(p.G), t1 = min(pc.L, pc.b_hi * kBlk);
  const uint8_t* v = static_cast<const uint8_t*>(p.d.v_cache);
#pragma unroll
  for (int e = 0; e < 4; ++e) sp[lane + 32 * e] = 255;
  bool apart = false;
  if (t0 < t1) {
#pragma unroll 1
    for (int j = max(t0, 0) / kP; j * kP < t1; j += kAhead) {
      const uint8_t* src[kAhead];
      uint4 x[kAhead][4 * kQ];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        src[k] = v + ((page_or_0(p, pc, j + k) * p.d.num_kv_heads + pc.h) * kD + lane) * kP * kEs;
#pragma unroll
        for (int e = 0; e < 4 * kQ; ++e)  // dims lane, + 32, ..
          x[k][e] = __ldg(reinterpret_cast<const uint4*>(src[k] + e / kQ * 32 * kP * kEs) + e % kQ);
      }
      uint32_t odd = 0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int e = 0; e < 4 * kQ; ++e)
          odd |= ((x[k][e].x & kOnes) + kLow) | ((x[k][e].y & kOnes) + kLow) |
                 ((x[k][e].z & kOnes) + kLow) | ((x[k][e].w & kOnes) + kLow);
      if ((odd & kSign) == 0) continue;
#pragma unroll 1
      for (int i = 0; i < kAhead * kP * 4; ++i) {  // one by one
        const int e = i & 3, t = j * kP + (i >> 2);
        if (t < t0 || t >= t1) continue;
        const uint8_t* at = (i >> 2 < kP ? src[0] : src[kAhead - 1]) + (e * 32 * kP + t % kP) * kEs;
        const uint32_t c = FP8 ? *at : *reinterpret_cast<const uint16_t*>(at);
        if ((c & kOnes & (FP8 ? 0xFFu : 0xFFFFu)) != (kOnes & (FP8 ? 0xFFu : 0xFFFFu))) continue;
        apart = true;
        if (t - t0 < sp[lane + 32 * e]) sp[lane + 32 * e] = (uint8_t)(t - t0);
      }
    }
  }
  return __any_sync(0xffffffffu, apart);
}

// The values of a piece that has some: one values warp's part of its blocks, u being the CTA's
// first.  False once a wait has run out.
template <bool FP8>
__device__ __noinline__ bool values_apart(const PrefillArgs& p, const Piece& pc, uint8_t* tiles,
                                          uint64_t* ready, uint64_t* room, uint32_t u,
                                          volatile int* abort_flag) {
  const int ct = threadIdx.x & 63, seen_all = pc.seen_all(p.G);
  const uint8_t* v = static_cast<const uint8_t*>(p.d.v_cache);
  for (int b = pc.b_lo; b < pc.b_hi; ++b, ++u) {
    if (u >= 2 && !wait_phase(&room[u & 1], (u >> 1) - 1, abort_flag, 4)) return false;
    uint8_t* dst = tiles + (u & 1) * kTileBytes;
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      // the thread's chunk i of 8 tokens of a dim, as the converters have it
      const int tok = b * kBlk + (FP8 ? (i >> 2) * kP + 8 * (i & 1) : 64 * (i >> 4) + 8 * (ct & 7));
      const uint32_t at = FP8 ? (i >> 4) * kHalf + ((i >> 1) & 1) * 8192 +
                                    (swz(ct, 0) ^ ((((i >> 1) & 6) + (i & 1)) << 4))
                              : (i >> 4) * kHalf + (i & 15) * 1024 + swz(ct >> 3, ct & 7);
      const int dim = FP8 ? ct + 64 * ((i >> 1) & 1) : 8 * (i & 15) + (ct >> 3);
      const long long ph = page_or_0(p, pc, tok / kP) * p.d.num_kv_heads + pc.h;
      const uint8_t* src = v + ((ph * kD + dim) * kP + tok % kP) * (FP8 ? 1 : 2);
      uint4 x;
      if (FP8) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(src));
        e4m3x4_to_f16(c.x, x.x, x.y);
        e4m3x4_to_f16(c.y, x.z, x.w);
      } else {
        x = __ldg(reinterpret_cast<const uint4*>(src));
      }
      uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t exp = (FP8 ? 0x7C00u : 0x7F80u) << (16 * (k & 1));
        if (tok + k >= pc.L || (tok + k >= seen_all && (y[k >> 1] & exp) == exp))
          y[k >> 1] &= 0xFFFFu << (16 * (~k & 1));
      }
      *reinterpret_cast<uint4*>(dst + at) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    fence_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ready[u & 1]);
  }
  return true;
}

struct Bars {
  uint64_t *k_ready, *k_free, *v_ready, *v_free;         // [2]
  uint64_t *q_ready, *q_free;
  uint64_t *s_full, *p_ready;                            // [tile][S buffer]
  uint64_t *pv_done, *o_full, *epi_done;                 // [tile]
  uint64_t *b_ml, *drain;
  uint64_t *ring_full, *ring_free, *sp_full;             // [kRing]
};

// --------------------------------------------------------------- kernel

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const Args a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(1024) uint8_t smem[];
  float4* meta = reinterpret_cast<float4*>(smem + OFF_META);
  float2* ml_b = reinterpret_cast<float2*>(smem + OFF_MLB);
  float* h_b = reinterpret_cast<float*>(smem + OFF_HB);
  uint8_t* spoil = smem + OFF_SPOIL;
  uint64_t* bp = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  Bars bar;
  bar.k_ready = bp, bar.k_free = bp + 2, bar.v_ready = bp + 4, bar.v_free = bp + 6;
  bar.q_ready = bp + 8, bar.q_free = bar.q_ready + 1;
  bar.s_full = bar.q_free + 1, bar.p_ready = bar.s_full + 4, bar.pv_done = bar.s_full + 8;
  bar.o_full = bar.pv_done + 2, bar.epi_done = bar.o_full + 2;
  bar.b_ml = bar.epi_done + 2, bar.drain = bar.b_ml + 1;
  bar.ring_full = bar.drain + 2, bar.ring_free = bar.ring_full + kRing;
  bar.sp_full = bar.ring_free + kRing;
  Piece* ring = reinterpret_cast<Piece*>(smem + OFF_RING);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);

  const PrefillArgs& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = p.d.num_kv_heads;
  const long long total = a.ws.pfx[a.V] * H;
  // at least a block's cost, so that every range holds a block's start
  const long long per = max((long long)kCostTwo, (total + a.grid - 1) / a.grid);
  const long long x_begin = (long long)blockIdx.x * per, x_end = min(total, x_begin + per);
  if (threadIdx.x == 0) a.ws.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (x_begin >= x_end) return;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (threadIdx.x == 64) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_ready[i], kConvWarps / 2);
      mbar_init(&bar.k_free[i], 2);  // (both tiles')
      mbar_init(&bar.v_ready[i], kConvWarps / 2);
      mbar_init(&bar.v_free[i], 2);
      mbar_init(&bar.pv_done[i], 1);
      mbar_init(&bar.o_full[i], 2);  // the products' end, and the issuing warp itself
      mbar_init(&bar.epi_done[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.s_full[i], 2);  // the products' end, and the issuing warp itself
      mbar_init(&bar.p_ready[i], 4);
    }
    mbar_init(bar.q_ready, kSoftWarps);
    mbar_init(bar.q_free, 2);
    mbar_init(bar.b_ml, 4);
    mbar_init(&bar.drain[0], 1);
    mbar_init(&bar.drain[1], 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar.ring_full[i], 1);
      mbar_init(&bar.sp_full[i], 1);
      mbar_init(&bar.ring_free[i], kMmaWarp + 2);  // every warp that reads it
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int32_t* ctl = p.d.ctl;
  bool go = true;  // the same in every lane of a warp
  auto wait = [&](uint64_t* b, uint32_t parity, int info) {
    if (go) go = wait_phase(b, parity, abort_flag, info);
    return go;
  };
  // the CTA's next piece (valid 0: none is left)
  Piece s;
  auto next_piece = [&](uint32_t piece) {
    const uint32_t k = piece % kRing;
    if (!wait(&bar.ring_full[k], piece / kRing, 1)) return false;
    const int4* w = reinterpret_cast<const int4*>(&ring[k]);
    const int4 w0 = w[0], w1 = w[1], w2 = w[2];
    s.r = w0.x, s.h = w0.y, s.row0 = w0.z, s.nrows = w0.w;
    s.b_lo = w1.x, s.b_hi = w1.y, s.nb = w1.z, s.L = w1.w;
    s.n = w2.x, s.q0 = w2.y, s.valid = w2.z;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.ring_free[k]);
    return s.valid != 0;
  };

  if (warp >= kSoftWarps && warp < kMmaWarp) {
    // ============================ converters ============================
    // Two warps have the keys, two the values: each goes at its own pace.
    const int cw = warp - kSoftWarps, ct = threadIdx.x & 63;
    const bool keys = cw < kConvWarps / 2;
    constexpr int kEs = FP8 ? 1 : 2;
    constexpr int kBatches = 2 * kEs;  // of 8 pieces of 16 bytes a thread, in a block's K or V
    constexpr long long kPageBytes = (long long)kP * kD * kEs;
    const uint8_t* cache = static_cast<const uint8_t*>(keys ? p.d.k_cache : p.d.v_cache);
    uint8_t* tiles = smem + (keys ? OFF_K : OFF_V);
    uint64_t *ready = keys ? bar.k_ready : bar.v_ready, *room = keys ? bar.k_free : bar.v_free;
    const uint32_t page_step = (uint32_t)(H * kPageBytes);
    // This thread's places in a swizzled tile.  e4m3: of its piece 2 q (16 codes, two chunks:
    // the other at ^ 16), piece 2 q + 1 `odd` bytes behind, a batch `turn`.  8 lanes hold a K
    // row, 4 of each half (those of the second store their chunks in the other order), or
    // 8 rows of V: no bank group is met twice.
    const bool swap = FP8 && keys && (ct & 4) != 0;
    const uint32_t odd = keys ? 1024 : 8192, turn = keys ? 8192 : kHalf;
    uint32_t off[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      off[q] = !FP8   ? swz(ct >> 3, ct & 7)
               : keys ? ((ct >> 2) & 1) * kHalf + swz(ct >> 3, 2 * (ct & 3) + swap) + q * 2048
                      : swz(ct, 2 * q);
    uint32_t u = 0;
    for (uint32_t piece = 0; next_piece(piece); ++piece) {
      // ---- the key blocks
      if (!keys) {
        if (!wait(&bar.sp_full[piece % kRing], piece / kRing, 16)) break;
        if (ring[piece % kRing].apart) {
          if (go) go = values_apart<FP8>(p, s, tiles, ready, room, u, abort_flag);
          if (!go) break;
          u += s.count();
          continue;
        }
      }
      const int32_t* prow = p.page_table + (long long)s.r * p.max_pages;
      const int npages = s.L / kP + (s.L % kP != 0);
      // lane l holds page l % 8 of a block: its id, -1 behind the request's
      // last page, -2 for an id out of range.  An id is looked at a block after
      // its load (page_raw), so that no load is waited for here.
      auto page_in = [&](int b) { return b < s.b_hi && b * kBlkPages + (lane & 7) < npages; };
      auto page_raw = [&](int b) -> int {
        return page_in(b) ? prow[b * kBlkPages + (lane & 7)] : 0;
      };
      auto page_of = [&](int raw, int b) -> int {
        return !page_in(b) ? -1 : raw >= 0 && raw < p.d.num_pages ? raw : -2;
      };
      auto scales_of = [&](int pg) -> float2 {  // of K and V
        if (!FP8 || cw != 0 || pg < 0) return make_float2(1.0f, 1.0f);
        const long long ph = (long long)pg * H + s.h;
        return make_float2(p.d.k_scale[ph], p.d.v_scale[ph]);
      };
      // A page that is not there (behind the length, or an id out of range) is read as
      // page 0: its scores are masked or its item is not written, and its V is
      // zeroed with what lies behind the length.
      const uint8_t* base = cache + s.h * kPageBytes;
      auto page_at = [&](int pgl, int l) {  // lane l's page
        const uint32_t pg = (uint32_t)__shfl_sync(0xffffffffu, max(pgl, 0), l);
        return base + (uint64_t)pg * page_step;
      };
      // Piece i of batch j, e4m3: the 16 bytes ct + 64 (i % 2) of page 4 j + i / 2:
      //   K token 8 (i % 2) + ct / 8 of the page, dims 16 (ct % 8) ..; V dim 64 (i % 2) + ct
      // bf16 (one chunk of a row in half j / 2):
      //   K token 64 (j % 2) + 8 i + ct / 8, dims 64 (j / 2) + 8 (ct % 8) ..
      //   V dim 64 (j % 2) + 8 i + ct / 8, tokens 64 (j / 2) + 8 (ct % 8) ..
      // A batch's registers are loaded with the next block's as soon as they are stored: as a
      // block is some 2,600 cycles, that is what it takes to have 32 KB in flight here.
      auto load = [&](int pgl, int j, uint4 (&x)[8]) {
        const uint8_t* src = nullptr;
        if (FP8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((i & 1) == 0) src = page_at(pgl, 4 * j + (i >> 1)) + ct * 16;
            x[i] = __ldg(reinterpret_cast<const uint4*>(src + (i & 1) * 1024));
          }
        } else if (keys) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((i & 1) == 0)
              src = page_at(pgl, 4 * (j & 1) + (i >> 1)) + (ct >> 3) * 256 + (ct & 7) * 16 +
                    (j >> 1) * 128;
            x[i] = __ldg(reinterpret_cast<const uint4*>(src + (i & 1) * 2048));
          }
        } else {
          src = page_at(pgl, 4 * (j >> 1) + ((ct & 7) >> 1)) + (j & 1) * 2048 + (ct >> 3) * 32 +
                (ct & 1) * 16;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(src + 256 * i));
        }
      };
      auto store = [&](uint8_t* dst, int j, const uint4 (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (FP8) {
            uint4 lo, hi;
            e4m3x4_to_f16(swap ? x[i].z : x[i].x, lo.x, lo.y);
            e4m3x4_to_f16(swap ? x[i].w : x[i].y, lo.z, lo.w);
            e4m3x4_to_f16(swap ? x[i].x : x[i].z, hi.x, hi.y);
            e4m3x4_to_f16(swap ? x[i].y : x[i].w, hi.z, hi.w);
            const uint32_t at = off[i >> 1] + j * turn + (i & 1) * odd;
            *reinterpret_cast<uint4*>(dst + at) = lo;
            *reinterpret_cast<uint4*>(dst + (at ^ 16)) = hi;
          } else {
            *reinterpret_cast<uint4*>(dst + off[0] + (j >> 1) * kHalf + (j & 1) * 8192 + 1024 * i) = x[i];
          }
        }
      };
      // tokens behind the length are zeroed where this thread stored them: their
      // bytes may be NaN, and 0 * NaN would reach the output
      auto clean_v = [&](uint8_t* dst, int b) {
        if ((b + 1) * kBlk <= s.L) return;
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {  // the thread's 16-byte chunks of 8 tokens
          const uint32_t at = FP8 ? (i >> 4) * kHalf + ((i >> 1) & 1) * 8192 +
                                        (swz(ct, 0) ^ ((((i >> 1) & 6) + (i & 1)) << 4))
                                  : (i >> 4) * kHalf + (i & 15) * 1024 + off[0];
          const int tok = FP8 ? (i >> 2) * kP + 8 * (i & 1) : 64 * (i >> 4) + 8 * (ct & 7);
          const int nv = s.L - b * kBlk - tok;  // valid tokens of the chunk
          if (nv >= 8) continue;
          uint16_t* h = reinterpret_cast<uint16_t*>(dst + at);
          for (int k = max(nv, 0); k < 8; ++k) h[k] = 0;
        }
      };
      // pages two blocks ahead are pulled into L2, 128 bytes a thread at a time (a bulk
      // prefetch's lanes are issued one after the other: 1,000 cycles for a block's pages)
      auto prefetch = [&](int pgl) {
#pragma unroll
        for (int i = 0; i < kBatches; ++i) {
          const int line = ct + 64 * i, pg = __shfl_sync(0xffffffffu, pgl, line / (16 * kEs));
          if (pg >= 0)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(base + (uint64_t)(uint32_t)pg * page_step +
                                                          line % (16 * kEs) * 128));
        }
      };
      // e4m3: an iteration before the first block loads it (one copy of the loads)
      const int b0 = s.b_lo - (FP8 ? 1 : 0);
      int raw2 = page_raw(b0 + 2);
      int pg0 = FP8 ? -1 : page_of(page_raw(b0), b0), pg1 = page_of(page_raw(b0 + 1), b0 + 1);
      uint4 x[2][8];
      float2 sc0 = make_float2(1.0f, 1.0f), sc1 = scales_of(pg1);
      if (!FP8) {
        load(pg0, 0, x[0]);
        load(pg0, 1, x[1]);
        prefetch(pg1);
      }
#pragma unroll 1
      for (int b = b0; b < s.b_hi; ++b) {
        const bool live = !FP8 || b >= s.b_lo;
        const uint32_t st = u & 1;
        const int pg2 = page_of(raw2, b + 2);
        raw2 = page_raw(b + 3);
        const float2 sc2 = scales_of(pg2);
        if (live && u >= 2 && !wait(&room[st], (u >> 1) - 1, keys ? 3 : 4)) break;
        uint8_t* dst = tiles + st * kTileBytes;
#pragma unroll
        for (int j = 0; j < kBatches; ++j) {
          if (live) store(dst, j, x[j & 1]);
          // (behind the last block: page 0, not used)
          if (j + 2 < kBatches) {
            if (live) load(pg0, j + 2, x[j & 1]);
          } else {
            load(pg1, j + 2 - kBatches, x[j & 1]);
          }
        }
        if (live) {
          if (!keys) clean_v(dst, b);
          if (cw == 0) {
            // (kept out of the arithmetic, where a masked score times NaN would be NaN)
            const bool odd = FP8 && !(sc0.x >= 0.0f && sc0.y >= 0.0f && sc0.x < INFINITY &&
                                      sc0.y < INFINITY);
            if (odd) sc0 = make_float2(1.0f, 1.0f);
            const float bias = __log2f(sc0.y);
            const uint32_t flags =
                (__any_sync(0xffffffffu, pg0 == -2) ? kBadPage : 0u) |
                (__any_sync(0xffffffffu, odd) ? kOdd : 0u) |
                (__any_sync(0xffffffffu, lane < kBlkPages && fabsf(bias) > 48.0f) ? kWide : 0u);
            if (lane < kBlkPages)
              meta[(u & (kMeta - 1)) * kBlkPages + lane] =
                  make_float4(sc0.x, bias, flags & kWide ? 0.0f : ex2(-bias),
                              __uint_as_float(flags | (odd ? kOddPage : 0u)));
            if (lane == 0 && (flags & kBadPage)) set_error(ctl, KV_ERR_BAD_PAGE_ID);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ready[st]);
          ++u;
        }
        prefetch(pg2);
        pg0 = pg1;
        pg1 = pg2;
        sc0 = sc1;
        sc1 = sc2;
      }
    }
  } else if (warp >= kMmaWarp) {
   if (warp < kMmaWarp + 2) {
    // ============================ MMA issuer ============================
    // One warp a tile.  Its units of a piece: n = 0, 1, ..; in an item of two tiles every
    // half block, in one of a single tile its own half of each block.  S of unit n + 1 is
    // issued before PV of unit n, so the tensor cores have work while P is awaited.
    const int x = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);
    const uint32_t leader = elect_one();
    // (a broadcast marks a value as the warp's own: the products take theirs from uniform
    // registers)
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    constexpr uint32_t kIdS = idesc(!FP8, kUnit), kIdPv = idesc(!FP8, kD);
    const uint64_t dq = sw128_desc(smem_u32(smem + OFF_Q), 16, 1024);
    const uint64_t dk = sw128_desc(smem_u32(smem + OFF_K), 16, 1024);
    const uint64_t dv = sw128_desc(smem_u32(smem + OFF_V), 16, 1024);
    int u0 = 0;               // the CTA's block at the piece's begin
    uint32_t t0 = 0;          // the tile's units before the piece
    for (uint32_t piece = 0; next_piece(piece); ++piece) {
      const bool both = s.both();
      const int cnt = s.count(), units = both ? 2 * cnt : cnt;
      const uint64_t q = dq + (uint32_t)((both ? x * kTileBytes : 0) >> 4);
      if (!wait(bar.q_ready, piece, 8)) break;
#pragma unroll 1
      for (int n = -1; n < units && go; ++n) {
        if (n + 1 < units) {  // ---- S of unit n + 1
          const int m = n + 1, u = u0 + (both ? m >> 1 : m), h = both ? m & 1 : x;
          const int st = __shfl_sync(0xffffffffu, u & 1, 0);
          const uint32_t b = __shfl_sync(0xffffffffu, 2 * x + ((t0 + m) & 1), 0);
          if ((h == 0 || !both) && !wait(&bar.k_ready[st], (uint32_t)(u >> 1), 9)) break;
          tc_fence_after();
          const uint64_t kk = dk + (uint32_t)((st * kTileBytes + h * (kHalf / 2)) >> 4);
          mma_ss4(leader, tm + 64 * b, q, kk, kIdS, 0);
          mma_ss4(leader, tm + 64 * b, q + (kHalf >> 4), kk + (kHalf >> 4), kIdS, 1);
          if (leader) {
            mma_commit(&bar.s_full[b]);
            mbar_arrive(&bar.s_full[b]);  // what this warp has waited for is seen behind it
            if (h == 1 || !both) mma_commit(&bar.k_free[st]);
            if (m == units - 1) mma_commit(bar.q_free);
          }
          __syncwarp();
        }
        if (n >= 0) {  // ---- O += P V of unit n
          const int u = u0 + (both ? n >> 1 : n), h = both ? n & 1 : x;
          const int st = __shfl_sync(0xffffffffu, u & 1, 0);
          const uint32_t b = __shfl_sync(0xffffffffu, 2 * x + ((t0 + n) & 1), 0);
          if ((h == 0 || !both) && !wait(&bar.v_ready[st], (uint32_t)(u >> 1), 6)) break;
          if (n == 0 && piece > 0 && !wait(&bar.epi_done[x], piece - 1, 7)) break;
          if (!wait(&bar.p_ready[b], (t0 + n) >> 1, 5)) break;
          tc_fence_after();
          const uint64_t vv = dv + (uint32_t)((st * kTileBytes + h * kHalf) >> 4);
          mma_ts4(leader, tm + tmem_o(x), tm + 64 * b, vv, kIdPv, n > 0 ? 1 : 0);
          if (!FP8) mma_ts4(leader, tm + tmem_o(x), tm + 64 * b + 32, vv, kIdPv, 1);
          if (leader) {
            mma_commit(&bar.pv_done[x]);
            if (h == 1 || !both) mma_commit(&bar.v_free[st]);
            if (n == units - 1) {
              mma_commit(&bar.o_full[x]);
              mbar_arrive(&bar.o_full[x]);
            }
          }
          __syncwarp();
        }
      }
      if (!go) break;
      u0 += cnt;
      t0 += units;
    }
    // every operation issued here finishes (bounded) before tensor memory is freed
    if (leader) {
      mma_commit(&bar.drain[x]);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&bar.drain[x], 0) && global_ns() - t0 < 100000000ull) {
      }
    }
    __syncwarp();
   } else {
    // ============================= scheduler =============================
    Walk c;
    {  // the last item that begins at or before x_begin, 32 entries a step
      int lo = 0, n = a.V;
      while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool le = lane * step < n && (lane == 0 || a.ws.pfx[at] * H <= x_begin);
        const int k = 31 - __clz((int)__ballot_sync(0xffffffffu, le));
        n = min(step, n - k * step);
        lo += k * step;
      }
      c.v = lo;
    }
    walk_item(c, a);
    c.h = (int)((x_begin - a.ws.pfx[c.v] * H) / c.cost());
    bool more = true;
    for (uint32_t piece = 0; more;) {
      walk_head(c, a, x_begin, x_end);
      if (c.s.b_lo < c.s.b_hi) {
        // the item that begins here and is cut by the range's end: for the combine
        if (lane == 0 && c.s.b_lo == 0 && c.s.b_hi < c.s.nb)
          a.ws.cut[blockIdx.x] = make_int4(
              c.v, c.h, (int)((c.blocks0() + (long long)c.s.w() * (c.s.nb - 1)) / per), 0);
        if (piece >= kRing && !wait(&bar.ring_free[piece % kRing], piece / kRing - 1, 10)) break;
        if (lane == 0) {
          ring[piece % kRing] = c.s;
          mbar_arrive(&bar.ring_full[piece % kRing]);
        }
        const bool apart = find_hidden<FP8>(p, c.s, spoil + piece % kRing * kD);
        if (lane == 0) {
          ring[piece % kRing].apart = apart;
          mbar_arrive(&bar.sp_full[piece % kRing]);
        }
        ++piece;
        // its query rows: the heads of a token lie together
        const int t0 = c.s.row0 / p.G, t1 = (c.s.row0 + c.s.nrows - 1) / p.G;
        for (int t = t0 + lane; t <= t1; t += 32)
          prefetch_l2(p.q + ((long long)(c.s.q0 + t) * p.Hq + c.h * p.G) * kD,
                      (uint32_t)(p.G * kD * 2));
      }
      if (c.x0 + c.cost() >= x_end) more = false;
      if (more && ++c.h == H) {
        c.h = 0;
        do {
          if (++c.v >= a.V) {
            more = false;
            break;
          }
        } while (a.ws.pfx[c.v + 1] == a.ws.pfx[c.v]);
        if (more) walk_item(c, a);
      }
      if (!more) {  // the end
        if (piece >= kRing && !wait(&bar.ring_free[piece % kRing], piece / kRing - 1, 10)) break;
        if (lane == 0) {
          ring[piece % kRing].valid = 0;
          mbar_arrive(&bar.ring_full[piece % kRing]);
        }
      }
    }
   }
  } else {
    // ============================== softmax ==============================
    // Scores in log2 units.  A page's V scale enters P as a bias log2(scale) on the
    // exponent, and M is the largest score + bias of a unit at which it was last taken (kRoom
    // below it), so that P stay below 2^15 whatever the scales.  The row sum l takes the bias
    // back out and has a reference R of its own: l counts tokens whose V scale is zero or tiny, for whose
    // scores M says nothing.  R is M as long as scales are near 1 (not kWide), else about the
    // largest score; it ends at l's own exponent, and O is brought to it.
    const int x = warp >> 2, row = (warp & 3) * 32 + lane;  // tile, row of the tile
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t to = tmem + tmem_o(x) + lanes;
    // phases of the barriers that this warp waits for, a bit each
    enum { kO = 2, kMl = 4, kOB = 8 };
    uint32_t u0 = 0, t = 0, ph = 0;  // the CTA's block at the piece's begin; units so far
    float next_qsc = 0.0f;
    // This thread's query row of piece k (-1: there is none) into the item's tile, and
    // the factor of its scores.  The two tiles' threads of an item with one tile hold the
    // same rows and store a half each.
    auto stage = [&](uint32_t k) {
      if (!wait(&bar.ring_full[k % kRing], k / kRing, 1)) return false;
      const volatile Piece* pc = ring + k % kRing;
      if (!pc->valid) return true;
      const int rows = pc->nrows, at = (rows > kTile ? x * kTile : 0) + row;
      const bool both = rows > kTile, live = at < rows;
      const bool any = __any_sync(0xffffffffu, live);
      const uint4* src = nullptr;
      float pw = 1.0f;
      if (any) {
        const int tg = pc->row0 + min(at, rows - 1), t = tg / p.G, g = tg - t * p.G;
        src = reinterpret_cast<const uint4*>(
            p.q + ((long long)(pc->q0 + t) * p.Hq + pc->h * p.G + g) * kD);
        next_qsc = fabsf(p.sm_scale_log2);
        if (FP8) {
          uint32_t mb = 0;
#pragma unroll 1
          for (int c = 0; c < 16; c += 8) {
            uint4 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __ldg(src + c + i);
#pragma unroll
            for (int i = 0; i < 8; ++i) mb = absbits_max8(mb, y[i]);
          }
          const int e = q_row_exp(max(mb & 0xFFFFu, mb >> 16));
          pw = pow2f(e);
          next_qsc *= pow2f(-e);
        }
      }
      // every product of the piece before has read the tiles
      if (k > 0 && !wait(bar.q_free, k - 1, 2)) return false;
      if (any) {
        const uint32_t flip = p.sm_scale_log2 < 0.0f ? 0x80008000u : 0u;  // the scale's sign
        uint8_t* dst = smem + OFF_Q + (both ? x * kTileBytes : 0);
#pragma unroll 1
        for (int j = both ? 0 : x; j < (both ? 2 : x + 1); ++j) {
          uint4 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __ldg(src + 8 * j + i);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint4 w = y[i];
            w.x ^= flip;
            w.y ^= flip;
            w.z ^= flip;
            w.w ^= flip;
            if (FP8) {
              w.x = bf16x2_to_f16x2_scaled(w.x, pw);
              w.y = bf16x2_to_f16x2_scaled(w.y, pw);
              w.z = bf16x2_to_f16x2_scaled(w.z, pw);
              w.w = bf16x2_to_f16x2_scaled(w.w, pw);
            }
            *reinterpret_cast<uint4*>(dst + j * kHalf + swz(row, i)) = w;
          }
        }
        fence_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar.q_ready);
      return true;
    };
    stage(0);
    for (uint32_t piece = 0;; ++piece) {
      const volatile Piece* pc = ring + piece % kRing;  // (stage has waited for it)
      if (!go || !pc->valid) break;
      const int rows = pc->nrows, cnt = pc->b_hi - pc->b_lo;
      const bool both = rows > kTile;
      const int tile0 = both ? x * kTile : 0;  // the tile's first row in the item
      const bool warp_live = tile0 + (warp & 3) * 32 < rows;
      // last positions that this row and the tile's first row see, from the piece's first
      // key block on
      const int seen0 = pc->L - pc->n - pc->b_lo * kBlk;
      const int lim = seen0 + (pc->row0 + min(tile0 + row, rows - 1)) / p.G;
      const int lim_all = seen0 + (pc->row0 + tile0) / p.G;
      const float qsc = next_qsc;
      float M = -INFINITY, l = 0.0f, R = -3e38f;
      // (in two steps: a factor below fp32's range may meet an l above 1)
      auto raise_R = [&](float to_ref) {
        const float f = ex2(0.5f * (R - to_ref));
        l = l * f * f;
        R = to_ref;
      };
      uint32_t flags = 0;
      const int units = both ? 2 * cnt : cnt;
#pragma unroll 1
      for (int n = 0; n < units; ++n, ++t) {
        const int i = both ? n >> 1 : n, h = both ? n & 1 : x;  // block of the piece, its half
        const int b = 2 * x + (t & 1);
        if (!wait(&bar.s_full[b], t >> 1, 11)) break;
        tc_fence_after();
        const float4* mt = meta + ((u0 + i) & (kMeta - 1)) * kBlkPages + kUnitPages * h;
        const uint32_t ts = tmem + 64 * b + lanes;
        if (warp_live) {
          const uint32_t fl = __float_as_uint(mt[0].w);
          flags |= fl;
          const int col0 = i * kBlk + h * kUnit;
          // P against the reference M as it is: as long as a row's P stay below 2^15 (their
          // sum tells) nothing is lost by a maximum that has grown since.  Only a first
          // unit, a row that has seen nothing yet, or a sum beyond that takes the unit's
          // maximum, and P again.
          bool take = n == 0 || __any_sync(0xffffffffu, M == -INFINITY);
          uint32_t pk[32], pl[FP8 ? 1 : 32];
          uint64_t add_l;
#pragma unroll 1
          for (;;) {
            float v[64];  // this row of S
            tmem_ld64(ts, v);
            if (lim_all < col0 + kUnit - 1) {  // columns <= lim are visible: the others to -inf
              const int c = lim - col0;
#pragma unroll
              for (int k = 0; k < kUnit; ++k) v[k] = k <= c ? v[k] : -INFINITY;
            }
            if (take) {
              float mx = -INFINITY;
#pragma unroll
              for (int g = 0; g < kUnitPages; ++g) {
                const float* w = &v[16 * g];
                float pm = fmaxf(w[0], w[1]);
#pragma unroll
                for (int k = 2; k < 16; k += 2) pm = fmaxf(fmaxf(pm, w[k]), w[k + 1]);
                // (a scale of 0 would make a masked score NaN)
                mx = FP8 ? fmaxf(mx, __fmaf_rn(pm, fmaxf(mt[g].x * qsc, 1e-37f), mt[g].y))
                         : fmaxf(mx, pm * fmaxf(qsc, 1e-37f));
              }
              float alpha = 1.0f;
              if (mx > M + 8.0f) {
                const float to = FP8 ? mx - kRoom : mx;
                alpha = M == -INFINITY ? 0.0f : ex2(M - to);
                if (!FP8) l *= alpha;
                M = to;
              }
              if (n > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                if (!wait(&bar.pv_done[x], t - 1, 12)) break;  // PV of the unit before
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < kD; c += 16) tmem_scale16(to + c, alpha);
              }
            }
            const float ref = M == -INFINITY ? 0.0f : M;
            uint64_t raw = 0;
#pragma unroll
            for (int g = 0; g < kUnitPages; ++g) {
              const float4 m = FP8 ? mt[g] : make_float4(1.0f, 0.0f, 1.0f, 0.0f);
              const float ks = fmaxf(FP8 ? m.x * qsc : qsc, 1e-37f), add = FP8 ? m.y - ref : -ref;
              const uint64_t k2 = pack2(ks, ks), a2 = pack2(add, add);
              uint64_t sum = 0;
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                float e0, e1;
                const float* w = &v[16 * g + k];
                unpack2(fma2(pack2(w[0], w[1]), k2, a2), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                sum = k == 0 ? pack2(e0, e1) : add2(sum, pack2(e0, e1));
                const uint32_t hi = pack_p<FP8>(e0, e1);
                pk[8 * g + k / 2] = hi;
                if (!FP8)
                  pl[(8 * g + k / 2) % (FP8 ? 1 : 32)] =
                      pack_p<false>(e0 - bf16_lo(hi), e1 - bf16_hi(hi));
              }
              raw = g == 0 ? sum : add2(raw, sum);
              if (FP8) {
                const uint64_t z = pack2(m.z, m.z);
                add_l = g == 0 ? mul2(sum, z) : fma2(sum, z, add_l);
              }
            }
            float r0, r1;
            unpack2(raw, r0, r1);
            if (!FP8) add_l = raw;
            if (take || !__any_sync(0xffffffffu, fmaxf(r0, r1) >= 32768.0f)) break;
            take = true;
          }
          if (!go) break;
          float s0, s1;
          unpack2(add_l, s0, s1);
          if (!FP8) l += s0 + s1;
          // where V scales lie far from 1, or M far above the scores, P can fall below fp32's
          // range while its weight counts: such a unit's sum is taken of the weights themselves
          const bool apart =
              FP8 && ((fl & kWide) || __any_sync(0xffffffffu, M - R > 40.0f && R > -1e38f));
          if (FP8 && !apart) {
            if (R < M) raise_R(M);
            l = __fmaf_rn(s0 + s1, ex2(M - R), l);
          }
          if (apart) {
#pragma unroll 1
            for (int c = 0; c < 2 * kUnitPages; ++c) {  // the unit twice: the largest, the sum
              const int g = c & (kUnitPages - 1);
              float y[16];
              tmem_ld16(ts + 16 * g, y);
              const float ks = fmaxf(mt[g].x * qsc, 1e-37f);
              float mx = -INFINITY;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                y[k] = col0 + 16 * g + k <= lim ? y[k] * ks : -INFINITY;
                mx = fmaxf(mx, y[k]);
              }
              if (c < kUnitPages) {
                if (mx > R + 8.0f) raise_R(mx);
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) l += ex2(y[k] - R);
              }
            }
          }
          if (FP8 && (fl & kOdd)) {  // a row that sees such a page becomes NaN
#pragma unroll 1
            for (int g = 0; g < kUnitPages; ++g)
              if ((__float_as_uint(mt[g].w) & kOddPage) && col0 + 16 * g <= lim)
                l = __int_as_float(0x7FFFFFFF);
          }
          tmem_st32u(ts, pk);
          if constexpr (!FP8) tmem_st32u(ts + 32, pl);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_ready[b]);
      }
      u0 += cnt;
      if (!go) break;
      if (!stage(piece + 1)) break;
      // ---- the piece's output
      float h = 1.0f;  // h^2: what brings O to R
      if (FP8) {
        if (l > 0.0f && l < INFINITY) {  // l to 1/2 .. 1, so that parts meet with what counts
          const int e = (int)(__float_as_uint(l) >> 23) - 126;
          l *= pow2f(-e);
          R += (float)e;
        }
        h = ex2(0.5f * (M - R));
        M = l == 0.0f ? -INFINITY : R;
      }
      // (a sum that is no number marks its part so: every part merged with it becomes NaN)
      if (l != l) M = INFINITY;
      const bool two = !both;  // A and B hold parts of the same rows
      if (!wait(&bar.o_full[x], (ph & kO) != 0, 13)) break;
      ph ^= kO;
      tc_fence_after();
      float wa = 1.0f, wb = 0.0f, hb = 1.0f;
      if (!both && x == 1) {  // B's part goes to A's warps
        ml_b[row] = make_float2(M, (flags & kBadPage) ? -1.0f : l);
        h_b[row] = h;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.b_ml);
      } else {
        if (two) {
          if (!wait(bar.b_ml, (ph & kMl) != 0, 14)) break;
          if (!wait(&bar.o_full[1], (ph & kOB) != 0, 15)) break;
          ph ^= kMl;
          tc_fence_after();
          const float2 b = ml_b[row];
          if (b.y < 0.0f) flags |= kBadPage;
          hb = h_b[row];
          const float Mn = fmaxf(M, b.x);
          // (-1: a part that saw nothing; its sum is 0)
          wa = M == -INFINITY ? -1.0f : ex2(M - Mn);
          wb = b.x == -INFINITY ? -1.0f : ex2(b.x - Mn);
          l = l * wa + b.y * wb;
          M = Mn;
        }
        ph ^= kOB;
        if (warp_live) {
          const bool bad = (flags & kBadPage) != 0, live = tile0 + row < rows;
          const bool whole = pc->b_lo == 0 && pc->b_hi == pc->nb;
          // zeros only for a row that sees no position: a sum of 0 or NaN goes into the output
          const bool none = lim < 0;  // (of a whole item: its first block is block 0)
          const float scale = 1.0f / l;
          const int slot = 2 * (int)blockIdx.x + (pc->b_lo > 0 ? 0 : 1), tg = pc->row0 + tile0 + row;
          const int t = tg / p.G, g = tg - t * p.G;
          const uint8_t* sp = spoil + piece % kRing * kD;
          const bool spoilt =
              __any_sync(0xffffffffu, reinterpret_cast<const uint32_t*>(sp)[lane] != 0xffffffffu);
          const int sees = t - pc->row0 / p.G - 1;  // the last of sp's tokens that this row sees
          uint16_t* out = p.out + ((long long)(pc->q0 + t) * p.Hq + pc->h * p.G + g) * kD;
          float4* part = a.ws.o + (long long)slot * 32 * kItemRows + tile0 + row;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[16];
            tmem_ld16(to + 16 * c, o);
            if (two) {
              float ob[16];
              tmem_ld16(tmem + tmem_o(1) + lanes + 16 * c, ob);
              // (a part that saw nothing holds zeros times whatever: leave it out)
#pragma unroll
              for (int k = 0; k < 16; ++k)
                o[k] = (wa != -1.0f ? o[k] * h * (h * wa) : 0.0f) +
                       (wb != -1.0f ? ob[k] * hb * (hb * wb) : 0.0f);
            } else if (FP8) {
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = o[k] * h * h;
            }
            if (spoilt) {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if ((int)sp[16 * c + k] <= sees) o[k] = __int_as_float(0x7FFFFFFF);
            }
            if (live && whole && !bad) {
#pragma unroll
              for (int k = 0; k < 16; k += 8) {
                uint4 y;
                y.x = pack_p<false>(o[k] * scale, o[k + 1] * scale);
                y.y = pack_p<false>(o[k + 2] * scale, o[k + 3] * scale);
                y.z = pack_p<false>(o[k + 4] * scale, o[k + 5] * scale);
                y.w = pack_p<false>(o[k + 6] * scale, o[k + 7] * scale);
                *reinterpret_cast<uint4*>(out + 16 * c + k) = none ? make_uint4(0, 0, 0, 0) : y;
              }
            } else if (live && !whole) {
#pragma unroll
              for (int k = 0; k < 16; k += 4)
                part[(4 * c + k / 4) * kItemRows] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            __syncwarp();  // the next tensor-memory load is the whole warp's
          }
          if (live && !whole)
            a.ws.ml[(long long)slot * kItemRows + tile0 + row] = make_float2(M, bad ? -1.0f : l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.epi_done[x]);
          if (two) mbar_arrive(&bar.epi_done[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ring_free[piece % kRing]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  if (threadIdx.x == 0 && *abort_flag != 0 &&
      atomicCAS(reinterpret_cast<int*>(ctl + KV_CTL_ERROR), 0, KV_ERR_TIMEOUT) == 0)
    ctl[KV_CTL_WAIT_INFO] = wait_info(kMmaWarp, 0, *abort_flag - 1);
}

// Cut items: the partials of the CTAs from the one that begins the item to the
// one that ends it, merged for 32 rows.
__global__ void __launch_bounds__(256) prefill_combine_kernel(const Args a) {
  pdl_wait();
  pdl_trigger();
  const int c0 = blockIdx.x;
  const int4 cut = a.ws.cut[c0];
  if (cut.x < 0) return;
  const PrefillArgs& p = a.p;
  const int4 it = a.ws.items[cut.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rr = blockIdx.y * 32 + lane;
  if (blockIdx.y * 32 >= it.z) return;
  __shared__ uint2 tile[32][33];
  __shared__ int skip[32];
  const bool live = rr < it.z;
  float M = -INFINITY, l = 0.0f;
  bool bad = false;
  auto slot_of = [&](int c) { return 2LL * c + (c == c0 ? 1 : 0); };
  if (live) {
    for (int c = c0; c <= cut.z; ++c) {
      const float2 ml = a.ws.ml[slot_of(c) * kItemRows + rr];
      bad = bad || ml.y < 0.0f;
      M = fmaxf(M, ml.x);
    }
  }
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0, 0, 0, 0);
  if (live && M != -INFINITY) {
    for (int c = c0; c <= cut.z; ++c) {
      const float2 ml = a.ws.ml[slot_of(c) * kItemRows + rr];
      if (ml.x == -INFINITY) continue;  // (saw nothing: zeros times whatever)
      const float w = exp2f(ml.x - M);
      l = __fmaf_rn(ml.y, w, l);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 o = a.ws.o[(slot_of(c) * 32 + warp + 8 * k) * kItemRows + rr];
        acc[k].x = __fmaf_rn(o.x, w, acc[k].x);
        acc[k].y = __fmaf_rn(o.y, w, acc[k].y);
        acc[k].z = __fmaf_rn(o.z, w, acc[k].z);
        acc[k].w = __fmaf_rn(o.w, w, acc[k].w);
      }
    }
  }
  // zeros only for a row that sees no position
  const int q0 = p.q_indptr[it.x];
  const bool none = p.seq_lens[it.x] - (p.q_indptr[it.x + 1] - q0) + (it.y + rr) / p.G < 0;
  const float inv = none ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    tile[lane][warp + 8 * k] = make_uint2(pack_p<false>(acc[k].x * inv, acc[k].y * inv),
                                          pack_p<false>(acc[k].z * inv, acc[k].w * inv));
  if (warp == 0) skip[lane] = !live || bad;
  __syncthreads();
  for (int i = warp; i < 32; i += 8) {
    if (skip[i]) continue;
    const int tg = it.y + blockIdx.y * 32 + i, t = tg / p.G, g = tg - t * p.G;
    *reinterpret_cast<uint2*>(p.out + ((long long)(q0 + t) * p.Hq + cut.y * p.G + g) * kD +
                              4 * lane) = tile[i][lane];
  }
}

}  // namespace

size_t prefill_ws_bytes(const kv_pool_desc& d, int B, int Hq, int total_q) {
  const int sms = sm_count();
  return sms > 0 ? ws_layout(nullptr, B, Hq / d.num_kv_heads, total_q, sms).bytes : 0;
}

cudaError_t launch_prefill(const PrefillArgs& p, cudaStream_t s, int* launches) {
  Args a;
  a.p = p;
  a.grid = sm_count();
  if (a.grid <= 0) return cudaErrorInvalidDevice;
  a.ws = ws_layout(p.workspace, p.B, p.G, p.total_q, a.grid);
  a.V = (int)item_count(p.B, p.G, p.total_q);
  const bool fp8 = p.d.dtype == KV_DTYPE_E4M3;
  cudaError_t e = fp8 ? cudaFuncSetAttribute(prefill_kernel<true>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)
                      : cudaFuncSetAttribute(prefill_kernel<false>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(prefill_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  e = fp8 ? launch_pdl(prefill_kernel<true>, dim3(a.grid), dim3(kThreads), kSmem, s, a)
          : launch_pdl(prefill_kernel<false>, dim3(a.grid), dim3(kThreads), kSmem, s, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  e = launch_pdl(prefill_combine_kernel, dim3(a.grid, kItemRows / 32), dim3(256), 0, s, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace kvfp8
