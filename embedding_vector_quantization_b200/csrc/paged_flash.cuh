// Attention of chunks of new tokens over paged caches on the tcgen05 tensor cores: d = 64 or 128, any MSE bits, with or
// without d signs, 16-bit queries.
//
// A chunk of n tokens reads each cached row n * G times (G query heads share a KV head), so each row is decoded once:
//   plan    one CTA lists the sequences that come here (more than `small_rows` query rows), their key tiles of 128 tokens
//           and their items of 256 query rows, with the running sum of the items' key tiles;
//   expand  key tiles -> f16 rows x_hat = Pi^T c[idx] + rnorm / norm * sqrt(pi/2) / m S^T (2 sigma - 1), as a
//           128 x d x 2 d contraction per tile on the tensor cores (with no signs Pi as an f16 pair); stored as the very shared-memory images the attention
//           wants, 32 KB a tile. Norms: a tile whose norms lie within 2^8 of each other has its rows times norm 2^-E, with
//           2^E >= every norm of it, which costs f16 nothing; any other tile ("apart") keeps rows of length about one, and the
//           attention multiplies scores and weights by the norms of its 128 tokens;
//   flash   softmax(scale q k^T) v over those tiles with the running maximum and sum of each row;
//   merge   items that several CTAs shared.
// Values come back in the original basis, so outputs need no rotation; keys times a Hadamard matrix, as the queries are: a
// channel far larger than the others would have its coordinate's rounding to f16 decide the scores, which the Hadamard matrix
// spreads over all coordinates. Signs cost no wider contraction: 4 d flops per (query row, key) for every format, where
// contracting the codes themselves would take 2 (2 d + m_k + m_v). The f16 rows are written and read once through L2 (512 B
// per token and head at d = 128).
//
// Roundings: c[idx] (hardly: table_factor in tq_api.cu), Pi with signs (an f16 pair without), S, rnorm / norm, x_hat, the
// prepared query (scaled by a power of two below 1) and the weights to f16 (11 bits; outputs have 8 or 11); every sum, maximum
// and exponent in fp32.
//
// Measured at 8 KV heads, 32 query heads, d = 128: a chunk of 1024 tokens over 32768 with signs takes 690 us (expansion 77,
// flash 570: 0.98 PFLOP/s, 0.60 of what a plain matrix product reaches); four prompts of up to 4096 tokens 380 us (flash 278).
// Nothing in the flash kernel is busy more than half the time (prompts: tensor pipe 43 % with the triangles' half tiles counted,
// issue slots 46 %, XU 35 %): it waits on each tile's chain of scores, maximum, barrier of 256 threads and weights.
#pragma once

#include <climits>

#include "encode_tc.cuh"
#include "paged_attn_simt.cuh"

namespace tqk {
namespace paged {

using etc::bar_arrive;
using etc::bulk_load;
using etc::expect_tx;
using etc::lds128;
using etc::named_sync;
using etc::sts128;
using etc::sw128_desc;
using etc::tc_fence_after;
using etc::tc_fence_before;
using etc::tmem_ld32;
using etc::tmem_wait_ld;
using etc::wait_bar;

constexpr int kKT = 128;          // tokens of a key tile
constexpr int kItemRows = 256;    // query rows of an item: two tiles of 128
constexpr int kItemCost = 3;      // an item's fixed cost in key tiles (query preparation, epilogue)
constexpr int kApart = 1 << 20;   // in place of an exponent: the tile's norms are apart from its rows
constexpr uint32_t kAtomRows = 128 * 128;   // 128 rows of 64 f16: one swizzle atom column

// Plan, in the workspace (ints): what plan_kernel writes.
struct Plan {
  int* head;         // [0] key tiles, [1] items, [2] units of one head, [3] the largest item's units
  int* tile_start;   // [B + 1] first key tile of a sequence
  int* item_start;   // [B + 1] first item of a sequence
  int* unit;         // [items + 1] running sum of the items' costs, within one head
  int* ke;           // [heads of a round][max_tiles] exponents of key tiles, or kApart
  int* ve;           // ... of value tiles
  float* kn;         // [heads of a round][max_tiles][128] norms of the key tiles that are kApart
  float* vn;         // ... of the value tiles
  uint32_t* seen;    // [max_tiles][4] tokens of the tile that exist and lie on a valid page
  uint8_t* krows;    // [heads of a round][max_tiles] f16 key tiles
  uint8_t* vrows;
  uint8_t* qrows;    // [heads of a round][max_items][2] f16 query tiles
  float* qfactor;    // [heads of a round][max_items][256] what a row's scores are multiplied by (log2), -1: it sees nothing
  float* part;       // [2 * CTAs][d / 4 + 1][256 rows] float4: results of cut items
  int max_tiles, max_items;
};

struct FlashArgs {
  const void* q;
  int64_t q_stride;
  int q_dtype, Hq, Hkv, G, head0, heads;   // the KV heads of this pass: head0 .. head0 + heads - 1
  Batch bt;
  Prep prep;
  Quant kq, vq;
  CacheView kc, vc;
  const uint8_t *kops, *vops;
  float scale;
  int causal, window, small_rows, ctas;
  Plan p;
  void* out;
  int* err;
};

__device__ __forceinline__ int seq_rows(const FlashArgs& a, int b) {
  const int n = seq_tokens(a.bt, b);
  return n * a.G > a.small_rows ? n : 0;   // tokens of the sequences that come here
}

// Keys [lo, hi) of tokens i0 .. i1 of sequence b, of n.
__device__ __forceinline__ void flash_range(const FlashArgs& a, int b, int i0, int i1, int n, int& lo, int& hi) {
  key_range(a.bt, b, i0, i1, n, a.causal, a.window, lo, hi);
}

constexpr int kPlanThreads = 1024;

// Exclusive running sum of v over the CTA, and the total.
__device__ __forceinline__ int block_scan(int v, int* warp_s, int& total) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int incl = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();
  if (lane == 31) warp_s[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = warp_s[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_s[lane] = w;
  }
  __syncthreads();
  total = warp_s[31];
  return incl - v + (warp ? warp_s[warp - 1] : 0);
}

// The last index i of start[0 .. n] with start[i] <= x, below n.
__device__ __forceinline__ int last_at_or_before(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same by a whole warp, 32 places at a time: two steps up to 1024 places.
__device__ __forceinline__ int warp_last_at_or_before(const int* start, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
    const int count = __popc(__ballot_sync(0xffffffffu, at < hi && start[at] <= x));   // start ascends: the first ones
    lo += max(0, count - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(FlashArgs a) {
  __shared__ int warp_s[32];
  const int tid = threadIdx.x;
  grid_dep_launch();
  int tiles = 0, items = 0, total;
  for (int b0 = 0; b0 < a.bt.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int nt = 0, ni = 0;
    if (b < a.bt.B) {
      const int n = seq_rows(a, b);
      if (seq_cut_short(a.bt, b)) report_error(a.err, kErrPaged);
      if (n > 0) {
        int lo, hi;
        flash_range(a, b, 0, n - 1, n, lo, hi);
        nt = hi > lo ? (hi + kKT - 1) / kKT - lo / kKT : 0;
        ni = (n * a.G + kItemRows - 1) / kItemRows;
      }
    }
    const int t = block_scan(nt, warp_s, total);
    const int tiles_now = total;
    const int i = block_scan(ni, warp_s, total);
    if (b < a.bt.B) a.p.tile_start[b] = tiles + t, a.p.item_start[b] = items + i;
    tiles += tiles_now, items += total;
  }
  if (tiles > a.p.max_tiles || items > a.p.max_items) {   // q_start is not ascending: nothing is computed
    if (tid == 0) {
      report_error(a.err, kErrPaged);
      a.p.head[0] = a.p.head[1] = a.p.head[2] = a.p.head[3] = 0;
    }
    grid_dep_wait();
    return;
  }
  if (tid == 0) a.p.tile_start[a.bt.B] = tiles, a.p.item_start[a.bt.B] = items;
  __syncthreads();
  int units = 0, most = 0;
  for (int i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int w = 0;
    if (i < items) {
      const int b = last_at_or_before(a.p.item_start, a.bt.B, i);
      const int n = seq_rows(a, b), row0 = (i - a.p.item_start[b]) * kItemRows;
      int lo, hi;
      flash_range(a, b, row0 / a.G, (min(n * a.G, row0 + kItemRows) - 1) / a.G, n, lo, hi);
      w = kItemCost + (hi > lo ? (hi + kKT - 1) / kKT - lo / kKT : 0);
    }
    const int u = block_scan(w, warp_s, total);
    if (i < items) a.p.unit[i] = units + u;
    units += total;
    most = max(most, w);
  }
  __shared__ int top_s;
  if (tid == 0) top_s = 0;
  __syncthreads();
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) atomicMax(&top_s, most);
  __syncthreads();
  if (tid == 0) {
    a.p.unit[items] = units;
    a.p.head[0] = tiles, a.p.head[1] = items, a.p.head[2] = units, a.p.head[3] = top_s;
  }
  grid_dep_wait();   // nothing here needs the kernel before (single tokens); what follows may count on it
}

// ---------------------------------------------------------------- expand

// Warps 0-7 write operands and 8-15 read results, in two groups each that take alternate tiles (and operand stages); 16 issues.
constexpr int kExThreads = 544;

template <int D>
struct ExLayout {
  static constexpr uint32_t kOpBytes = 2 * (D / 64) * D * 128;          // Pi^T and S^T, K-major
  // operand rows of 128 tokens: two stages of codes and signs, or four of codes alone
  static constexpr uint32_t kABytes = 4 * (D / 64) * kAtomRows;
  static constexpr uint32_t kA = kOpBytes;
  static constexpr uint32_t kLut = kA + kABytes;                        // 32 KB
  static constexpr uint32_t kScale = kLut + 32768;                      // float [4][128]
  static constexpr uint32_t kBars = kScale + 2048;                      // op_full, a_full[4], a_empty[4], d_full[4], d_empty[4]
  static constexpr uint32_t kMisc = kBars + 17 * 8;                     // tmem slot, abort, extremes[2 groups][2][8]
  static constexpr uint32_t kBytes = kMisc + 8 + 128;
};
static_assert(ExLayout<128>::kBytes <= 232448, "expand layout exceeds the shared memory of one CTA");

// Loads that stay where they are written: ahead of the work on the row before (left to itself, the compiler puts them off to
// where they are used, and every tile waits for memory).
__device__ __forceinline__ uint2 load_ahead64(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_ahead32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint16_t load_ahead16(const void* p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];\n" : "=h"(v) : "l"(p));
  return v;
}

// One token's packed row, loaded ahead.
template <int D>
struct Row {
  uint32_t code[D / 8];   // 4 bits: all of them
  uint32_t sign[D / 32];
  uint32_t norm;          // as loaded (fp16 or fp32): nothing here waits for a load
  uint16_t rnorm;
  bool ok;
};

template <int D>
__device__ __forceinline__ void load_row(const Quant& Q, const CacheView& c, int64_t at, Row<D>& r) {
  r.ok = at >= 0;
  r.norm = 0, r.rnorm = 0;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) r.code[i] = 0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) r.sign[i] = 0;
  if (at < 0) return;
  if (Q.norm_dtype == TQ_F16) r.norm = load_ahead16(static_cast<const __half*>(c.norms) + at);
  else r.norm = load_ahead32(static_cast<const float*>(c.norms) + at);
  const uint2* w = reinterpret_cast<const uint2*>(c.codes + at * Q.codes_B);   // rows are multiples of 8 bytes
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    if (8 * i < Q.codes_B) {
      const uint2 v = load_ahead64(w + i);
      r.code[2 * i] = v.x, r.code[2 * i + 1] = v.y;
    }
  if (Q.m > 0) {
    const uint2* s = reinterpret_cast<const uint2*>(c.signs + at * Q.signs_B);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint2 v = load_ahead64(s + i);
      r.sign[2 * i] = v.x, r.sign[2 * i + 1] = v.y;
    }
    if (Q.bits > 0) r.rnorm = load_ahead16(c.rnorms + at);
  }
}

// Table of f16 centroids (times cent_up, which brings them next to f16's values) for one packed byte (3 bits: for one pair of fields), a copy for each bank so that no two lanes
// of a phase meet: 4 bits 4 B x 32 copies, 2 bits 8 B x 16, 1 bit 16 B x 8, 3 bits 64 pairs x 32.
__device__ __forceinline__ void build_lut(const Quant& Q, uint8_t* lut, int tid, int nthreads) {
  if (Q.bits == 0) return;
  // a warp per entry, a lane per word: lane l writes the pair l mod (words of an entry)
  const int per = Q.bits == 3 ? 2 : 8 / Q.bits, n = Q.bits == 3 ? 64 : 256, mask = (1 << Q.bits) - 1;
  const int lane = tid & 31, p = (lane & (per / 2 - 1)) * 2 * Q.bits;
  const uint32_t own = __half_as_ushort(__float2half_rn(lane <= mask ? Q.cent[lane] * Q.cent_up : 0.f));   // lane i: centroid i
  for (int v = tid >> 5; v < n; v += nthreads >> 5) {
    const uint32_t x = __shfl_sync(0xffffffffu, own, v >> p & mask), y = __shfl_sync(0xffffffffu, own, v >> (p + Q.bits) & mask);
    *reinterpret_cast<uint32_t*>(lut + v * 128 + 4 * lane) = x | y << 16;
  }
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// Table entries: the table does not change once it is built, so these need not stay in order (in order, each product would
// wait for its own entries before the next ones are asked for).
__device__ __forceinline__ uint32_t table32(uint32_t a) {
  uint32_t v;
  asm("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 table64(uint32_t a) {
  uint2 v;
  asm("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 table128(uint32_t a) {
  uint4 v;
  asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// (w >> 8 i & 255) * 128: byte i as a table offset, one shift and one mask
__device__ __forceinline__ uint32_t byte128(uint32_t w, int i) { return (i == 0 ? w << 7 : w >> (8 * i - 7)) & 0x7f80u; }

// Chunk c (8 coordinates, 16 bytes of f16) of a row's codes.
template <int D>
__device__ __forceinline__ uint4 code_chunk(const Row<D>& r, int bits, int c, uint32_t lut, int lane) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (bits == 4) {
    const uint32_t w = r.code[c], b = 4 * lane;
    v = make_uint4(table32(lut + (byte128(w, 0) | b)), table32(lut + (byte128(w, 1) | b)), table32(lut + (byte128(w, 2) | b)),
                   table32(lut + (byte128(w, 3) | b)));
  } else if (bits == 2) {
    const uint32_t w = r.code[c >> 1], b = 8 * (lane & 15);
    const uint2 x = table64(lut + (byte128(w, 2 * (c & 1)) | b)), y = table64(lut + (byte128(w, 2 * (c & 1) + 1) | b));
    v = make_uint4(x.x, x.y, y.x, y.y);
  } else if (bits == 1) {
    v = table128(lut + 16 * (lane & 7) + (((r.code[c >> 2] >> (8 * (c & 3))) & 255u) << 7));
  } else if (bits == 3) {   // 24 bits from bit 24 c on
    const int w0 = (24 * c) >> 5, sh = (24 * c) & 31;
    const uint32_t x = __funnelshift_r(r.code[w0], r.code[min(w0 + 1, D / 8 - 1)], sh), b = lut + 4 * lane;
    v = make_uint4(table32(b + ((x & 63u) << 7)), table32(b + ((x >> 6 & 63u) << 7)), table32(b + ((x >> 12 & 63u) << 7)),
                   table32(b + ((x >> 18 & 63u) << 7)));
  }
  return v;
}

// Places 8 c .. 8 c + 7 of a row's signs: place 32 u + 2 i holds the sign of projection 32 u + i, place 32 u + 2 i + 1 that
// of 32 u + 16 + i (one shift and one mask give both halves of a word); the rows of S^T in the operand follow that order.
template <int D>
__device__ __forceinline__ uint4 sign_chunk(const Row<D>& r, int c, uint32_t ratio2) {
  const uint32_t w = ~r.sign[c >> 2];
  const int i = 4 * (c & 3);
  auto two = [&](int k) { return ((k < 16 ? w << (15 - k) : 0u) & 0x80008000u) ^ ratio2; };
  return make_uint4(two(i), two(i + 1), two(i + 2), two(i + 3));
}

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
__device__ __forceinline__ void bulk_store_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_store_wait() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// f16 x f16, fp32 sums, M = 128; bn: B is MN-major (its N runs along the bytes)
__host__ __device__ constexpr uint32_t flash_idesc(int N, bool bn) {
  return (1u << 4) | (bn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// ---- issue by one lane of a whole warp: the warp stays together, so that addresses and descriptors live in uniform
// registers (a lone thread spends longer on moving them there than the tensor cores on the instruction)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %0, 0;\n setp.ne.u32 p, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n}\n" ::"r"(leader),
      "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0));
}
// A in tensor memory (lane = row, 8 columns of two f16 per 16 K).
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %0, 0;\n setp.ne.u32 p, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n}\n" ::"r"(leader),
      "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void commit_one(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %0, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}\n" ::"r"(leader),
      "r"(bar)
      : "memory");
}

// Where a CTA's walk over (head, key tile) pairs stands; the sequence is looked up only when the tile leaves it.
struct TileCursor {
  int h, tile, b, first, last, base, lo, hi;   // tiles [first, last) of sequence b; key 0 of tile `first` is at `base`, keys are [lo, hi)
};
__device__ __forceinline__ void cursor_seek(const FlashArgs& a, int tiles, TileCursor& c, int step) {
  c.tile += step;
  while (c.tile >= tiles) c.tile -= tiles, ++c.h;
  if (c.tile >= c.first && c.tile < c.last) return;
  c.b = warp_last_at_or_before(a.p.tile_start, a.bt.B, c.tile);
  c.first = a.p.tile_start[c.b], c.last = a.p.tile_start[c.b + 1];
  const int n = seq_rows(a, c.b);
  flash_range(a, c.b, 0, n - 1, n, c.lo, c.hi);
  c.base = c.lo / kKT * kKT;
}

// Grid: 2 x CTAs; even CTAs keys, odd CTAs values; CTA j of the n of a kind takes pairs [j W / n, (j + 1) W / n) of W.
template <int D>
__global__ void __launch_bounds__(kExThreads, 1) paged_expand_kernel(FlashArgs a) {
  using L = ExLayout<D>;
  extern __shared__ __align__(1024) unsigned char smem_tiles[];
  unsigned char* const smem = smem_tiles;
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kind = blockIdx.x & 1, j0 = blockIdx.x >> 1, step = gridDim.x >> 1;
  const Quant& Q = kind ? a.vq : a.kq;
  const CacheView& C = kind ? a.vc : a.kc;
  const uint32_t bars = base + L::kBars;
  const uint32_t op_full = bars;
  auto a_full = [&](int s) { return bars + 8u * (1 + s); };
  auto a_empty = [&](int s) { return bars + 8u * (5 + s); };
  auto d_full = [&](int s) { return bars + 8u * (9 + s); };
  auto d_empty = [&](int s) { return bars + 8u * (13 + s); };
  const int NS = Q.m > 0 ? 2 : 4;                                      // stages: tile i uses i mod NS
  const uint32_t stage_bytes = L::kABytes / NS;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  uint32_t* extremes = reinterpret_cast<uint32_t*>(smem + L::kMisc + 8);
  float* scale_s = reinterpret_cast<float*>(smem + L::kScale);
  if ((base & 1023u) != 0) {
    if (tid == 0) report_error(a.err, kErrInternal);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + L::kBars);
    bar_init(b, 1);
    for (int s = 0; s < 4; ++s) bar_init(b + 1 + s, 4), bar_init(b + 5 + s, 1), bar_init(b + 9 + s, 1), bar_init(b + 13 + s, 4);
  }
  build_lut(Q, smem + L::kLut, tid, kExThreads);
  grid_dep_wait();
  grid_dep_launch();   // only now: the next kernel reads the plan too
  const int tiles = a.p.head[0];
  const int64_t work = (int64_t)tiles * a.heads;
  const int w0 = (int)(work * j0 / step), mine = (int)(work * (j0 + 1) / step) - w0;
  if (mine == 0) return;
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(base + L::kMisc), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (*abort_flag || wait_bar(bar, parity)) return;
    *abort_flag = 1;
    report_error(a.err, kErrTimeout);
  };
  constexpr int katoms = 2 * (D / 64);   // 64-wide slices of the contraction: codes and signs, or codes twice

  if (warp < 8) {
    // ---- operand rows: thread = token of the tile. Under way at a time: the page of the token after next, the next row.
    const int g = warp >> 2, r = tid & 127;
    const float down = 1.f / Q.cent_up;   // the tables' factor, out again
    uint32_t* const extremes_g = extremes + 16 * g;
    TileCursor c{(int)(w0 / tiles), (int)(w0 % tiles), 0, 0, 0, 0, 0, 0};
    // The cursor's token: its page as loaded (nothing waits for it yet), and where in the page.
    struct Spot {
      int page, slot, h, tile;
      bool in;
    };
    auto spot = [&]() -> Spot {
      Spot p;
      const int pos = c.base + (c.tile - c.first) * kKT + r;
      p.in = pos >= c.lo && pos < c.hi, p.h = c.h, p.tile = c.tile;   // pages behind the window may be someone else's
      const uint32_t pi = (uint32_t)pos / (uint32_t)a.bt.page_size;
      p.slot = pos - (int)pi * a.bt.page_size;
      p.page = p.in ? (int)load_ahead32(a.bt.table + (int64_t)c.b * a.bt.max_pages + pi) : -1;
      return p;
    };
    auto row_of = [&](const Spot& p) -> int64_t {   // -1: bad page, -2: not among the keys
      if (!p.in) return -2;
      if (p.page < 0 || p.page >= a.bt.num_pages) return -1;
      return ((int64_t)p.page * a.Hkv + a.head0 + p.h) * a.bt.page_size + p.slot;
    };
    Row<D> cur, nxt;
    Spot s0{-1, 0, 0, 0, false}, s1 = s0;   // this group's next tile, and the one after
    int64_t at0 = -2;
    if (g < mine) {
      cursor_seek(a, tiles, c, g);
      s0 = spot();
      at0 = row_of(s0);
      load_row<D>(Q, C, at0, nxt);
    }
    if (g + 2 < mine) {
      cursor_seek(a, tiles, c, 2);
      s1 = spot();
    }
    for (int i = g; i < mine; i += 2) {
      const int s = i % NS;
      cur = nxt;
      const int64_t here = at0;
      const int tile = s0.tile, h = s0.h;
      s0 = s1;
      if (i + 2 < mine) {
        at0 = row_of(s0);
        load_row<D>(Q, C, at0, nxt);
      }
      if (i + 4 < mine) {
        cursor_seek(a, tiles, c, 2);
        s1 = spot();
      }
      float norm = Q.norm_dtype == TQ_F16 ? __half2float(__ushort_as_half((uint16_t)cur.norm)) : __uint_as_float(cur.norm);
      if (here == -1) report_error(a.err, kErrPaged);
      const unsigned there = __ballot_sync(0xffffffffu, cur.ok);
      if (kind == 0 && h == 0 && lane == 0) a.p.seen[4 * tile + (warp & 3)] = there;
      float ratio = 1.f;   // of the residual norm to the norm
      if (Q.m > 0 && Q.bits > 0) {
        ratio = norm != 0.f ? __half2float(__ushort_as_half(cur.rnorm)) / norm : 0.f;
        ratio *= Q.cent_up;
        if (!(fabsf(ratio) <= 65504.f)) {   // the row stays finite, its norm tells that it is not
          ratio = 0.f;
          if (fabsf(norm) < INFINITY) norm = NAN;
        }
      }
      // the tile's largest and smallest norm other than 0: as bits, which are ordered like them (NaN above all)
      const uint32_t bits = cur.ok ? __float_as_uint(norm) & 0x7fffffffu : 0u;
      const uint32_t top_w = __reduce_max_sync(0xffffffffu, bits), low_w = __reduce_min_sync(0xffffffffu, bits ? bits : 0xffffffffu);
      uint32_t* const ext = extremes_g + (i & 2) * 4;   // two sets in turn: one barrier a tile is enough
      if (lane == 0) ext[warp & 3] = top_w, ext[4 + (warp & 3)] = low_w;
      named_sync(1 + g, 128);
      const uint32_t top = max(max(ext[0], ext[1]), max(ext[2], ext[3])), low = min(min(ext[4], ext[5]), min(ext[6], ext[7]));
      // Above a quotient of 2^8 the smallest rows would lose digits to f16's least exponent, which norms apart cost none.
      const bool apart = top >= 0x7f800000u || (top > 0 && top - low > 8u << 23);
      int e = -126;
      if (top > 0) frexpf(__uint_as_float(top), &e);
      e = max(-126, min(126, e));
      if (i >= NS) wait(a_empty(s), (i / NS - 1) & 1);
      scale_s[s * 128 + r] = !cur.ok ? 0.f : down * (apart ? 1.f : ldexpf(norm, -e));
      if (r == 0) (kind ? a.p.ve : a.p.ke)[(int64_t)h * a.p.max_tiles + tile] = apart ? kApart : e;
      if (apart) (kind ? a.p.vn : a.p.kn)[((int64_t)h * a.p.max_tiles + tile) * kKT + r] = cur.ok ? norm : 0.f;
      const uint32_t row = base + L::kA + s * stage_bytes + r * 128;
      if (Q.bits > 0) {
#pragma unroll
        for (int ch = 0; ch < D / 8; ++ch) {
          const uint4 v = code_chunk<D>(cur, Q.bits, ch, base + L::kLut, lane);
          sts128(row + (ch >> 3) * kAtomRows + (((ch & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < D / 8; ++ch) sts128(row + (ch >> 3) * kAtomRows + (((ch & 7) ^ (r & 7)) << 4), 0, 0, 0, 0);
      }
      if (Q.m > 0) {
        const uint32_t r2 = half2_bits(ratio, ratio);
#pragma unroll
        for (int ch = 0; ch < D / 8; ++ch) {
          const uint4 v = sign_chunk<D>(cur, ch, r2);
          sts128(row + (D / 64 + (ch >> 3)) * kAtomRows + (((ch & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(a_full(s));
    }
  } else if (warp < 16) {
    // ---- results: thread = token; the row goes out through the operand stage that produced it
    const int g = (warp >> 2) & 1, r = tid & 127;
    for (int i = g; i < mine; i += 2) {
      const int s = i % NS, h = (w0 + i) / tiles, tile = (w0 + i) - h * tiles;
      wait(d_full(s), (i / NS) & 1);
      tc_fence_after();
      const float f = scale_s[s * 128 + r];
      const uint32_t row = base + L::kA + s * stage_bytes + r * 128;
#pragma unroll 1
      for (int c4 = 0; c4 < D / 32; ++c4) {
        uint32_t v[32];
        tmem_ld32(tmem + s * 128 + ((uint32_t)((warp & 3) * 32) << 16), v, 32 * c4);
        tmem_wait_ld(v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            o[x] = half2_bits(__uint_as_float(v[8 * k + 2 * x]) * f, __uint_as_float(v[8 * k + 2 * x + 1]) * f);
          const int c = 4 * c4 + k;
          sts128(row + (c >> 3) * kAtomRows + (((c & 7) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before();
      fence_async();
      named_sync(3 + g, 128);
      if (r == 0) {
        const uint32_t bytes = (D / 64) * kAtomRows;
        uint8_t* dst = (kind ? a.p.vrows : a.p.krows) + ((int64_t)h * a.p.max_tiles + tile) * bytes;
        bulk_store(dst, base + L::kA + s * stage_bytes, bytes);
        bulk_store_read_wait();
        bar_arrive(a_empty(s));
      }
      if (lane == 0) bar_arrive(d_empty(s));
    }
    if (r == 0) bulk_store_wait();
  } else {
    // ---- contraction
    const uint32_t lead = elect_one();
    constexpr uint32_t kAtomOp = D * 128;
    if (lead) {
      expect_tx(op_full, katoms * kAtomOp);
      for (int k = 0; k < katoms; ++k) bulk_load(base + k * kAtomOp, (kind ? a.vops : a.kops) + k * kAtomOp, kAtomOp, op_full);
    }
    wait(op_full, 0);
    const uint64_t a_desc = sw128_desc(base + L::kA), b_desc = sw128_desc(base);
    for (int i = 0; i < mine; ++i) {
      const int s = i % NS;
      wait(a_full(s), (i / NS) & 1);
      if (i >= NS) wait(d_empty(s), (i / NS - 1) & 1);
      tc_fence_after();
      const uint64_t ad = a_desc + ((s * stage_bytes) >> 4);
      for (int k = 0; k < katoms; ++k)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int ka = Q.m > 0 ? k : k & (D / 64 - 1);
          const uint64_t x = ad + ((ka * kAtomRows + kk * 32) >> 4), y = b_desc + ((k * kAtomOp + kk * 32) >> 4);
          if (k == 0 && kk == 0) mma_ss<false>(lead, tmem + s * 128, x, y, flash_idesc(D, false));
          else mma_ss<true>(lead, tmem + s * 128, x, y, flash_idesc(D, false));
        }
      commit_one(lead, d_full(s));
    }
    // tensor memory is released below: the last contractions must have ended
    for (int i = max(0, mine - NS); i < mine; ++i) (void)wait_bar(d_full(i % NS), (i / NS) & 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u) : "memory");
}

// ---------------------------------------------------------------- queries

// Query rows to f16 tiles, as the attention wants them in shared memory: norm, rotation, then times the power of two that
// brings every coordinate below one. Four lanes per row; lane q of them holds the 16-byte chunks q, q + 4, ...: the partners
// of a rotation of the whole head (half a head away) are its own. Bound by latency and bytes: as many rows in flight as fit.
// Grid: (max_items * 8, heads): 32 rows per CTA, small enough to run beside the expansion's CTAs: it is started when all of
// those run, which have seen the plan complete, and needs nothing of theirs.
constexpr int kQtThreads = 128;
template <int D>
__global__ void __launch_bounds__(kQtThreads) paged_qtile_kernel(FlashArgs a) {
  constexpr int C = D / 32;   // chunks per lane
  const int item = blockIdx.x >> 3, h = blockIdx.y;
  grid_dep_launch();
  if (item >= a.p.head[1] && (item | h) > 0) return;
  const int ql = threadIdx.x & 3, r = (blockIdx.x & 7) * 32 + (threadIdx.x >> 2);
  const int rot = a.prep.cos_sin ? a.prep.rot_dim : 0, half = rot >> 1;
  const bool f16 = a.q_dtype == TQ_F16;
  if (item >= a.p.head[1]) {   // no item at all
    grid_dep_wait();
    return;
  }
  const int b = warp_last_at_or_before(a.p.item_start, a.bt.B, item), n = seq_rows(a, b);
  const int64_t t0 = a.bt.q_start[b], slot = (int64_t)h * a.p.max_items + item;
  const int pos0 = a.bt.len[b] - n, row = (item - a.p.item_start[b]) * kItemRows + r;
  const bool live = row < n * a.G;
  const int tok = live ? row / a.G : 0, g = live ? row - tok * a.G : 0, hq = (a.head0 + h) * a.G + g;
  int64_t rp = pos0 + tok;
  bool ok = live;
  if (live && rot) {
    if (a.prep.pos) rp = a.prep.pos[t0 + tok];
    if (rp < 0 || rp >= a.prep.max_pos) {
      if (ql == 0 && (a.prep.pos || rp >= 0)) report_error(a.err, kErrPaged);
      ok = false;
    }
  }
  const uint16_t* src = static_cast<const uint16_t*>(a.q) + (t0 + tok) * a.q_stride + (int64_t)hq * D;
  const float* cs_row = a.prep.cos_sin + rp * rot;
  float z[8 * C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint4 w = ok ? __ldg(reinterpret_cast<const uint4*>(src) + ql + 4 * c) : make_uint4(0, 0, 0, 0);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = f16 ? etc::pair_to_float2<true>(x[e]) : etc::pair_to_float2<false>(x[e]);
      z[8 * c + 2 * e] = v.x, z[8 * c + 2 * e + 1] = v.y;
    }
  }
  float rms = 1.f;
  if (a.prep.weight) {
    float ss = 0.f;
#pragma unroll
    for (int x = 0; x < 8 * C; ++x) ss = fmaf(z[x], z[x], ss);
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    rms = rsqrtf(ss / (float)D + a.prep.eps);
    const bool many = !(ss < kManySquares);
    if (__any_sync(0xffffffffu, many)) {
      float s2 = 0.f;
#pragma unroll
      for (int x = 0; x < 8 * C; ++x) s2 = fmaf(z[x] * kSmaller, z[x] * kSmaller, s2);
      s2 += __shfl_xor_sync(0xffffffffu, s2, 1);
      s2 += __shfl_xor_sync(0xffffffffu, s2, 2);
      if (many) rms = kSmaller * rsqrtf(s2 / (float)D);
    }
#pragma unroll
    for (int x = 0; x < 8 * C; ++x) z[x] *= rms * load_any(a.prep.weight, a.prep.weight_dtype, 8 * (ql + 4 * (x >> 3)) + (x & 7));
  }
  float top = 0.f;
#pragma unroll
  for (int x = 0; x < 8 * C; ++x) top = fmaxf(top, fabsf(z[x]));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (ok && rot == D && !a.prep.interleaved) {
#pragma unroll
    for (int c = 0; c < C / 2; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k0 = 8 * (ql + 4 * c) + 4 * e;
        const float4 co = *reinterpret_cast<const float4*>(cs_row + k0);
        const float4 si = *reinterpret_cast<const float4*>(cs_row + D / 2 + k0);
        const float cc[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float& lo = z[8 * c + 4 * e + x];
          float& hi = z[8 * (c + C / 2) + 4 * e + x];
          const float p = lo, w = hi;
          lo = p * cc[x] - w * sn[x], hi = w * cc[x] + p * sn[x];
        }
      }
  } else if (ok && rot) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k0 = 8 * (ql + 4 * c) + 2 * e;
        float& y0 = z[8 * c + 2 * e];
        float& y1 = z[8 * c + 2 * e + 1];
        if (k0 < rot && a.prep.interleaved) {
          const float co = cs_row[k0 >> 1], si = cs_row[half + (k0 >> 1)], p = y0, w = y1;
          y0 = p * co - w * si, y1 = w * co + p * si;
        } else if (k0 < rot) {   // the partner may be any lane's: read again
          const int kk = k0 < half ? k0 : k0 - half, other = k0 < half ? k0 + half : k0 - half;
          const float sg = k0 < half ? -rms : rms;
          float p0 = load_any(src, a.q_dtype, other), p1 = load_any(src, a.q_dtype, other + 1);
          if (a.prep.weight) {
            p0 *= load_any(a.prep.weight, a.prep.weight_dtype, other);
            p1 *= load_any(a.prep.weight, a.prep.weight_dtype, other + 1);
          }
          y0 = y0 * cs_row[kk] + sg * p0 * cs_row[half + kk];
          y1 = y1 * cs_row[kk + 1] + sg * p1 * cs_row[half + kk + 1];
        }
      }
  }
  // the power of two that brings every coordinate below one; a rotation makes none larger than 2^(1/2) times the largest
  int e = 0;
  if (top > 0.f && top < INFINITY) frexpf(top, &e);
  e = max(-126, min(126, e + 1));
  // Coordinates below one, then times the Hadamard matrix (over the bits of the coordinate's number: three within a chunk, two of
  // the lane, the rest of the chunk), as the keys' rows are.
  const float sc = a.scale < 0.f ? -ldexpf(1.f, -e) : ldexpf(1.f, -e);
  if (ql == 0) a.p.qfactor[slot * kItemRows + r] = ok || !live ? ldexpf(fabsf(a.scale) * (0.125f * 1.44269504089f), e) : -1.f;
#pragma unroll
  for (int x = 0; x < 8 * C; ++x) z[x] *= sc;
#pragma unroll
  for (int w = 1; w < 8 * C; w *= 2)
#pragma unroll
    for (int x = 0; x < 8 * C; ++x)
      if (!(x & w)) {
        const float p = z[x], o = z[x + w];
        z[x] = p + o, z[x + w] = p - o;
      }
#pragma unroll
  for (int w = 1; w < 4; w *= 2) {
    const float sign = ql & w ? -1.f : 1.f;
#pragma unroll
    for (int x = 0; x < 8 * C; ++x) z[x] = fmaf(sign, z[x], __shfl_xor_sync(0xffffffffu, z[x], w));
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int ch = ql + 4 * c;
    *reinterpret_cast<uint4*>(a.p.qrows + ((2 * slot + (r >> 7)) * (D / 64) + (ch >> 3)) * kAtomRows + (r & 127) * 128 +
                              (((ch & 7) ^ (r & 7)) << 4)) =
        make_uint4(half2_bits(z[8 * c], z[8 * c + 1]), half2_bits(z[8 * c + 2], z[8 * c + 3]),
                   half2_bits(z[8 * c + 4], z[8 * c + 5]), half2_bits(z[8 * c + 6], z[8 * c + 7]));
  }
  if (item == 0 && h == 0) grid_dep_wait();   // what follows may count on the expansion: this kernel ends behind it
}

// ---------------------------------------------------------------- flash

// Warps 0-15: softmax, two threads per query row (warps 0-3 and 4-7: keys 0-63 and 64-127 of the rows of query tile 0, 8-15
// of tile 1): with one thread per row its chain of loads, maximum and exponentials took twice the time that the tensor cores
// need for the other tile. 16: copies; 17: MMAs; 18, 19 fill their warpgroup, which gives registers up:
// 640 threads x 96 at launch = 128 x (4 x 104 + 64).
constexpr int kFlThreads = 640;
constexpr int kFlStages = 4;      // ring of key and value tiles, in the order K0 V0 K1 V1 ...

template <int D>
struct FlLayout {
  static constexpr uint32_t kTile = (D / 64) * kAtomRows;   // 32 KB: 128 rows of D f16
  static constexpr uint32_t kQ = 0;                         // two query tiles
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kBars = kRing + kFlStages * kTile;
  // full[4], empty[4], q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], o_free[2]
  static constexpr int kNumBars = 2 * kFlStages + 12;
  static constexpr uint32_t kRow = kBars + 8 * kNumBars;     // float2 [2][256]: what the two threads of a row tell each other
  static constexpr uint32_t kMisc = kRow + 4096;
  static constexpr uint32_t kBytes = kMisc + 16;
};
static_assert(FlLayout<128>::kBytes <= 232448, "flash layout exceeds the shared memory of one CTA");

// MN-major operand (N along the 128-byte rows, one row per K index): blocks of 64 N are kAtomRows apart, groups of 8 K
// indices 1024 bytes.
__device__ __forceinline__ uint64_t mn_desc16(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(kAtomRows >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// CTA c of P takes units [c U / P, (c + 1) U / P) of the round's U = heads * units, head by head, item by item.
struct Span {
  int64_t u0, u1;
};
__device__ __forceinline__ Span span_of(int64_t U, int c, int P) {
  if (U <= 0x1fffff && P < 2047) {   // 32-bit quotients do
    const uint32_t u = (uint32_t)U, p = (uint32_t)P;
    return {u * (uint32_t)c / p, u * (uint32_t)(c + 1) / p};
  }
  return {U * c / P, U * (c + 1) / P};
}

// What CTA c does: its even share, or one whole item where every item has a CTA and the largest is at most kWholeSlack key
// tiles above the share (about 2.4 us each at d = 128: less than writing, reading and merging cut items takes).
constexpr int kWholeSlack = 8;
__device__ __forceinline__ bool whole_items(const FlashArgs& a) {
  const int items = a.p.head[1], P = a.ctas;
  const int64_t U = (int64_t)a.p.head[2] * a.heads;
  return (int64_t)items * a.heads <= P && a.p.head[3] <= U / P + kWholeSlack;
}
__device__ __forceinline__ Span flash_span(const FlashArgs& a, int c) {
  const int items = a.p.head[1], units = a.p.head[2];
  if (!whole_items(a)) return span_of((int64_t)units * a.heads, c, a.ctas);
  if (c >= items * a.heads) return {0, 0};
  const int h = c / items, i = c - h * items;
  return {(int64_t)h * units + a.p.unit[i], (int64_t)h * units + a.p.unit[i + 1]};
}

// A CTA's share of one item: key tiles [t0, t1) of nt. Found by whole warps.
struct Segment {
  int h, item, b, n, row0, nrows, lo_tile, nt, t0, t1;
  int64_t next;   // first unit after the item
  int64_t first;  // first unit of the item
};
__device__ __forceinline__ Segment segment_at(const FlashArgs& a, int items, int units, int64_t u, int64_t u1) {
  Segment s;
  s.h = (int)(u / units);
  const int r = (int)(u - (int64_t)s.h * units);
  s.item = warp_last_at_or_before(a.p.unit, items, r);
  s.first = (int64_t)s.h * units + a.p.unit[s.item];
  s.next = (int64_t)s.h * units + a.p.unit[s.item + 1];
  s.b = warp_last_at_or_before(a.p.item_start, a.bt.B, s.item);
  s.n = seq_rows(a, s.b);
  s.row0 = (s.item - a.p.item_start[s.b]) * kItemRows;
  s.nrows = min(kItemRows, s.n * a.G - s.row0);
  int lo, hi, lo_all, hi_all;
  flash_range(a, s.b, s.row0 / a.G, (s.row0 + s.nrows - 1) / a.G, s.n, lo, hi);
  flash_range(a, s.b, 0, s.n - 1, s.n, lo_all, hi_all);
  (void)hi_all;
  s.nt = (int)(s.next - s.first) - kItemCost;
  s.lo_tile = lo / kKT - lo_all / kKT;   // relative to the sequence's first tile
  s.t0 = max(0, (int)(u - s.first) - kItemCost);
  s.t1 = max(0, (int)(min(u1, s.next) - s.first) - kItemCost);
  return s;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr), "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
      "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// ---- pairs of fp32 values in one 64-bit register: one instruction for two sums or products
__device__ __forceinline__ uint64_t pair2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
// 2^x for two values on the fused multiply-add pipe (the exponential unit alone would bind the kernel: 16 results a cycle
// against 4096 fused multiply-adds of the tensor cores). x = n + f, |f| <= 1/2; 2^f by the cubic of least relative error
// (7.5e-5, a sixth of what the rounding to f16 costs; fitted by linear programming over [-1/2, 1/2]); n is added to the
// exponent. x <= -126 gives a value near 2^-126, which becomes 0 in f16.
__device__ __forceinline__ float2 exp2_poly(float x, float y) {
  const uint64_t v = pair2(fmaxf(x, -126.f), fmaxf(y, -126.f));
  const uint64_t big = pair2(12582912.f, 12582912.f), none = pair2(-12582912.f, -12582912.f), neg = pair2(-1.f, -1.f);
  const uint64_t t = add2(v, big);               // 1.5 2^23: the integer part lands in the low bits
  const uint64_t f = fma2(add2(t, none), neg, v);
  uint64_t p = fma2(f, pair2(0.055171772837638855f, 0.055171772837638855f), pair2(0.2426113784313202f, 0.2426113784313202f));
  p = fma2(p, f, pair2(0.6932609677314758f, 0.6932609677314758f));
  p = fma2(p, f, pair2(0.9999279975891113f, 0.9999279975891113f));
  const float2 q = unpair2(p), n = unpair2(t);
  return make_float2(__int_as_float(__float_as_int(q.x) + (__float_as_int(n.x) << 23)),
                     __int_as_float(__float_as_int(q.y) + (__float_as_int(n.y) << 23)));
}
// Barrier of n threads that tells whether any of them said so.
__device__ __forceinline__ bool bar_any(int id, int n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
// Of so many pairs of exponentials one goes to the polynomial: 579 us with a fourth for a chunk of 1024 tokens over 32768
// (8 KV heads, 32 query heads, d = 128), 577 with a third, 597 with half and 584 without; four prompts 276, 274, 282 and 281.
constexpr int kPolyEvery = 4;

template <int D>
__global__ void __launch_bounds__(kFlThreads, 1) paged_flash_kernel(FlashArgs a) {
  using L = FlLayout<D>;
  extern __shared__ __align__(1024) unsigned char smem_tiles[];
  unsigned char* const smem = smem_tiles;
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_launch();
  grid_dep_wait();
  const int items = a.p.head[1], units = a.p.head[2];
  const Span sp = flash_span(a, blockIdx.x);
  if ((base & 1023u) != 0) {
    if (tid == 0) report_error(a.err, kErrInternal);
    return;
  }
  if (sp.u0 >= sp.u1) return;
  const uint32_t bars = base + L::kBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kFlStages + s); };
  auto q_full = [&](int i) { return bars + 8u * (2 * kFlStages + i); };
  auto q_empty = [&](int i) { return bars + 8u * (2 * kFlStages + 2 + i); };
  auto s_full = [&](int i) { return bars + 8u * (2 * kFlStages + 4 + i); };
  auto p_full = [&](int i) { return bars + 8u * (2 * kFlStages + 6 + i); };
  auto pv_done = [&](int i) { return bars + 8u * (2 * kFlStages + 8 + i); };
  auto o_free = [&](int i) { return bars + 8u * (2 * kFlStages + 10 + i); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  if (tid == 0) {
    *abort_flag = 0;
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + L::kBars);
    for (int x = 0; x < L::kNumBars; ++x) {   // p_full and o_free: a query tile's eight warps; the others: one copy or commit
      const int y = x - 2 * kFlStages;
      bar_init(b + x, y == 6 || y == 7 || y == 10 || y == 11 ? 8 : 1);
    }
  }
  if (warp == 17) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(base + L::kMisc), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t col_s[2] = {tmem, tmem + 128}, col_o[2] = {tmem + 256, tmem + 384};
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (*abort_flag || wait_bar(bar, parity)) return;
    *abort_flag = 1;
    report_error(a.err, kErrTimeout);
  };

  if (warp == 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    int k = 0, seg = 0;   // tiles issued (keys and values counted apart), segments with tiles
    for (int64_t u = sp.u0; u < sp.u1;) {
      const Segment s = segment_at(a, items, units, u, sp.u1);
      u = s.next;
      if (s.t1 <= s.t0) continue;
      if (lane == 0) {
        const int64_t t = (int64_t)s.h * a.p.max_tiles + a.p.tile_start[s.b] + s.lo_tile;
        for (int j = s.t0; j < s.t1; ++j)
          for (int kv = 0; kv < 2; ++kv, ++k) {
            const int st = k % kFlStages;
            if (k >= kFlStages) wait(empty(st), (k / kFlStages - 1) & 1);
            if (*abort_flag) break;
            expect_tx(full(st), L::kTile);
            bulk_load(base + L::kRing + st * L::kTile, (kv ? a.p.vrows : a.p.krows) + (t + j) * L::kTile, L::kTile, full(st));
            if (j == s.t0 && kv == 0) {   // the queries, behind the first keys
              const int64_t qt = 2 * ((int64_t)s.h * a.p.max_items + s.item);
              for (int i = 0; i < 2; ++i) {
                if (seg > 0) wait(q_empty(i), (seg - 1) & 1);
                if (*abort_flag) break;
                expect_tx(q_full(i), L::kTile);
                bulk_load(base + L::kQ + i * L::kTile, a.p.qrows + (qt + i) * L::kTile, L::kTile, q_full(i));
              }
              ++seg;
            }
          }
      }
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;   // the whole warp, or its next search would wait for a lane
    }
    if (lane == 0) {
      // never leave with a copy still landing in this CTA's shared memory
      for (int i = max(0, k - kFlStages); i < k; ++i) (void)wait_bar(full(i % kFlStages), (i / kFlStages) & 1);
      if (seg > 0)
        for (int i = 0; i < 2; ++i) (void)wait_bar(q_full(i), (seg - 1) & 1);
    }
  } else if (warp == 17) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    const uint32_t lead = elect_one();
    const uint64_t q_desc = sw128_desc(base + L::kQ), k_desc = sw128_desc(base + L::kRing), v_desc = mn_desc16(base + L::kRing);
    constexpr uint32_t kT16 = L::kTile >> 4;   // a tile in the descriptors' unit of 16 bytes
    int k = 0, seg = 0, tile = 0;   // ring position, segments with tiles, tiles
    for (int64_t u = sp.u0; u < sp.u1;) {
      const Segment s = segment_at(a, items, units, u, sp.u1);
      u = s.next;
      const int nt = s.t1 - s.t0;
      if (nt <= 0) continue;
      auto scores = [&](int i, int kk, bool last) {   // S_i = Q_i K^T
        const uint64_t qd = q_desc + i * kT16, kd = k_desc + (kk % kFlStages) * kT16;
        mma_ss<false>(lead, col_s[i], qd, kd, flash_idesc(128, false));
#pragma unroll
        for (int c = 1; c < D / 16; ++c) {
          const uint32_t off = ((c >> 2) * kAtomRows + (c & 3) * 32) >> 4;
          mma_ss<true>(lead, col_s[i], qd + off, kd + off, flash_idesc(128, false));
        }
        commit_one(lead, s_full(i));
        if (last) commit_one(lead, q_empty(i));
      };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        wait(q_full(i), seg & 1);
        if (i == 0) wait(full(k % kFlStages), (k / kFlStages) & 1);
        tc_fence_after();
        scores(i, k, nt == 1);
      }
      commit_one(lead, empty(k % kFlStages));
      for (int j = 0; j < nt; ++j, k += 2, ++tile) {
        const int vs = (k + 1) % kFlStages;
        const uint64_t vd = v_desc + vs * kT16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 0) wait(full(vs), ((k + 1) / kFlStages) & 1);
          if (j == 0 && seg > 0) wait(o_free(i), (seg - 1) & 1);
          wait(p_full(i), tile & 1);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 8; ++c)   // 16 tokens at a time
            mma_ts(lead, col_o[i], col_s[i] + 8 * c, vd + ((c * 2048) >> 4), flash_idesc(D, true), c > 0 ? 1u : (j > 0 ? 1u : 0u));
          commit_one(lead, pv_done(i));
          if (i == 1) commit_one(lead, empty(vs));
          if (j + 1 < nt) {
            if (i == 0) {
              wait(full((k + 2) % kFlStages), ((k + 2) / kFlStages) & 1);
              tc_fence_after();
            }
            scores(i, k + 2, j + 2 == nt);
            if (i == 1) commit_one(lead, empty((k + 2) % kFlStages));
          }
        }
      }
      ++seg;
    }
    // tensor memory is released below: the last contractions must have ended
    if (tile > 0)
      for (int i = 0; i < 2; ++i) (void)wait_bar(pv_done(i), (tile - 1) & 1);
  } else if (warp >= 18) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
    // ---- softmax: thread = half a query row
    const int i = warp >> 3, half = (warp >> 2) & 1, r = tid & 127;
    float2* const mine = reinterpret_cast<float2*>(smem + L::kRow) + 256 * i + 128 * half + r;
    const float2* const theirs = reinterpret_cast<float2*>(smem + L::kRow) + 256 * i + 128 * (half ^ 1) + r;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t cs = col_s[i] + lanes, co = col_o[i] + lanes + half * (D / 2);   // scores; this thread's value sums
    int tile = 0;   // tiles of this CTA so far
    for (int64_t u = sp.u0; u < sp.u1;) {
      const Segment s = segment_at(a, items, units, u, sp.u1);
      const bool first_unit = u == s.first;
      u = s.next;
      const int nt = s.t1 - s.t0;
      const int row = s.row0 + 128 * i + r;
      const bool live = 128 * i + r < s.nrows;
      const int tok = live ? row / a.G : 0, g = live ? row - tok * a.G : 0;
      const int64_t t = (int64_t)a.bt.q_start[s.b] + tok;
      const int hq = (a.head0 + s.h) * a.G + g;
      const int64_t oat = (t * a.Hq + hq) * D;
      if (nt <= 0) {
        if (s.nt == 0 && first_unit && live) {   // no key at all
          uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + oat + half * (D / 2));
          for (int c = 0; c < D / 16; ++c) o[c] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      const int len = max(0, a.bt.len[s.b]), cap = (int)min((int64_t)len, (int64_t)a.bt.max_pages * a.bt.page_size);
      const int pos = a.bt.len[s.b] - s.n + tok;
      int lo = 0, hi = live ? cap : 0;   // keys this row sees
      if (a.causal) {
        hi = min(hi, pos + 1);
        if (a.window > 0) lo = max(0, pos - a.window + 1);
      }
      const float factor = a.p.qfactor[((int64_t)s.h * a.p.max_items + s.item) * kItemRows + 128 * i + r];
      const float qscale = fabsf(factor);
      if (factor < 0.f) hi = 0;   // no rotation for its position: the row sees nothing
      // ---- key tiles
      const int tile0 = a.p.tile_start[s.b] + s.lo_tile;
      const int64_t te = (int64_t)s.h * a.p.max_tiles + tile0;
      int lo_all, hi_all;
      flash_range(a, s.b, 0, s.n - 1, s.n, lo_all, hi_all);
      const int key_first = (lo_all / kKT + s.lo_tile) * kKT;
      // Running reference (log2) and sum of the weights. The value sums have a unit of their own, 2^(m + b), which follows what the
      // row's weights and the value tiles' exponents make together: a large value that the row hardly sees costs it nothing.
      // Where b is set it is a whole number, so that a row's largest weight comes out as a power of two, exact in f16; where m
      // moves, b makes up for it (sums that kept to whole numbers would have to be scaled then: 562 -> 609 us). limit: what a
      // score may be without moving m (-infinity while there is no unit; NaN where |m| is above 2^14, whose tiles all take the
      // rare part below); rest: -(m + b), or 0.
      float m = -INFINITY, l = 0.f, b = -INFINITY, limit = -INFINITY, rest = 0.f;
      int ke = a.p.ke[te + s.t0], ve = a.p.ve[te + s.t0];
      uint4 seen = *reinterpret_cast<const uint4*>(a.p.seen + 4 * (tile0 + s.t0));
      for (int j = s.t0; j < s.t1; ++j, ++tile) {
        const bool k_apart = ke == kApart, v_apart = ve == kApart;
        const float ev = (float)ve;
        float c = fmaxf(qscale * exp2f((float)ke), 1e-37f);   // above 0: c times the mask's -infinity stays -infinity
        const uint4 seen_now = seen;
        if (j + 1 < s.t1) {
          ke = a.p.ke[te + j + 1], ve = a.p.ve[te + j + 1];
          seen = *reinterpret_cast<const uint4*>(a.p.seen + 4 * (tile0 + j + 1));
        }
        const int k0 = key_first + j * kKT + 64 * half;
        const uint32_t there[2] = {half ? seen_now.z : seen_now.x, half ? seen_now.w : seen_now.y};
        const bool whole = (there[0] & there[1]) == 0xffffffffu && k0 >= lo && k0 + 64 <= hi;
        const bool masked = __any_sync(0xffffffffu, !whole);
        wait(s_full(i), tile & 1);
        tc_fence_after();
        uint32_t v[2][32];
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) tmem_ld32(cs + 64 * half, v[q4], 32 * q4);
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) tmem_wait_ld(v[q4]);
        if (masked) {
#pragma unroll
          for (int q4 = 0; q4 < 2; ++q4) {
            const int f = k0 + 32 * q4, lo1 = min(max(lo - f, 0), 32), hi1 = min(max(hi - f, 0), 32);
            const uint32_t ok = there[q4] & (hi1 >= 32 ? 0xffffffffu : (1u << hi1) - 1u) & (lo1 >= 32 ? 0u : 0xffffffffu << lo1);
#pragma unroll
            for (int x = 0; x < 32; ++x) v[q4][x] = ok >> x & 1 ? v[q4][x] : 0xff800000u;
          }
        }
        float mx4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t(&w)[32] = v[q >> 1];
          const int x0 = 16 * (q & 1);
          mx4[q] = __uint_as_float(w[x0]);
#pragma unroll
          for (int x = 1; x < 15; x += 2) mx4[q] = max_nan(mx4[q], __uint_as_float(w[x0 + x]), __uint_as_float(w[x0 + x + 1]));
          mx4[q] = max_nan(mx4[q], __uint_as_float(w[x0 + 15]));
        }
        float top = max_nan(max_nan(mx4[0], mx4[1], mx4[2]), mx4[3]) * c;
        float rv = ev + rest;         // weights in the sums' unit: 2^(c score + rv)
        const float gap = b - ev;     // from those to the sum's weights, log2
        bool odd = false;             // rv and the sum of weights are made in the rare part below
        // The reference moves only when a score exceeds it by 2^8, the unit when a product of weight and value norm exceeds it by
        // 2^12: weights stay within f16, and the sums are rarely scaled. All threads of the tile learn here whether any row moves;
        // from here on no score is needed in tensor memory. (A NaN moves them, and the row is NaN from there on.) Rare as well:
        // tiles whose norms are apart; values so small that the weights would be too small to add up; scores so large that their
        // products with c have to be rounded before the reference is taken off, as the reference was.
        if (bar_any(1 + i, 256, k_apart || v_apart || !(top <= limit && top + rv <= 12.f && gap <= 40.f))) {
          if (k_apart) {
            const float4* n = reinterpret_cast<const float4*>(a.p.kn + (te + j) * kKT + 64 * half);
            c = 1.f, top = -INFINITY;
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float4 w4 = n[x];
              const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t& y = v[x >> 3][4 * (x & 7) + k];
                if (y != 0xff800000u) y = __float_as_uint(__uint_as_float(y) * (w[k] * qscale));   // (masked)
                top = max_nan(top, __uint_as_float(y));
              }
            }
          }
          // the largest weight times value norm, log2, relative to this half's largest weight
          float top_o = ev, sum = 0.f;
          const float top_ref = top == -INFINITY ? 0.f : top;
          if (v_apart) {   // from here on scores are relative to this half's largest and have their value norm with them; the sum is without
            const float4* n = reinterpret_cast<const float4*>(a.p.vn + (te + j) * kKT + 64 * half);
            top_o = -INFINITY;
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float4 w4 = n[x];
              const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t& y = v[x >> 3][4 * (x & 7) + k];
                const float s1 = __fmul_rn(__uint_as_float(y), c) - top_ref, s2 = s1 == -INFINITY ? s1 : s1 + lg2(w[k]);
                sum += ex2(s1);
                top_o = max_nan(top_o, s2);
                y = __float_as_uint(s2);
              }
            }
          }
          *mine = make_float2(top, top_o);
          named_sync(1 + i, 256);
          const float2 other = *theirs;
          const float both = max_nan(top, other.x);
          if (!(both <= m + 8.f)) {
            if (m > -INFINITY) l *= ex2(m - both), b += m - both;
            m = both;
          }
          const float most = m == -INFINITY ? -INFINITY : max_nan((top - m) + top_o, (other.x - m) + other.y);
          float f = 1.f;
          if (!(most <= b + 12.f)) {
            const float now = ceilf(most);
            if (b > -INFINITY) f = ex2(b - now);   // (sums without a unit are zeros)
            b = now;
          }
          if (j > s.t0 && __any_sync(0xffffffffu, f != 1.f)) {
            wait(pv_done(i), (tile - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int q4 = 0; q4 < D / 64; ++q4) {
              uint32_t y[32];
              tmem_ld32(co, y, 32 * q4);
              tmem_wait_ld(y);
#pragma unroll
              for (int x = 0; x < 32; ++x) y[x] = __float_as_uint(__uint_as_float(y[x]) * f);
              tmem_st16(co + 32 * q4, y);
              tmem_st16(co + 32 * q4 + 16, y + 16);
            }
          }
          named_sync(1 + i, 256);   // the exchanged maxima have been read
          const float m_ref = m == -INFINITY ? 0.f : m, b_ref = b == -INFINITY ? 0.f : b;
          rest = b == -INFINITY ? 0.f : -(m + b);
          limit = b == -INFINITY ? -INFINITY : fabsf(m) <= 16384.f ? m + 8.f : NAN;
          rv = ev + rest;
          if (v_apart) {
            odd = true, c = 1.f, rv = (top_ref - m_ref) - b_ref, sum *= ex2(top_ref - m_ref);
          } else if (__any_sync(0xffffffffu, b - ev > 40.f || fabsf(m_ref) > 16384.f)) {
            odd = true, rv = ev - b_ref;
#pragma unroll
            for (int x = 0; x < 64; ++x) {
              uint32_t& y = v[x >> 5][x & 31];
              const float s1 = __fmul_rn(__uint_as_float(y), c) - m_ref;
              sum += ex2(s1);
              y = __float_as_uint(s1);
            }
            c = 1.f;
          }
          l += m == -INFINITY ? 0.f : sum;
        }
        const uint64_t c2 = pair2(c, c), r2 = pair2(rv, rv);
        uint64_t sums[2] = {0, 0};
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {
          uint32_t p[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float2 e = unpair2(fma2(pair2(__uint_as_float(v[q4][2 * x]), __uint_as_float(v[q4][2 * x + 1])), c2, r2));
            const float2 w = x % kPolyEvery == kPolyEvery - 1 ? exp2_poly(e.x, e.y) : make_float2(ex2(e.x), ex2(e.y));
            sums[x & 1] = add2(sums[x & 1], pair2(w.x, w.y));
            p[x] = half2_bits(w.x, w.y);
          }
          // the weights of 128 keys take the first 64 columns of the scores
          tmem_st16(cs + 32 * half + 16 * q4, p);
        }
        const float2 sum2 = unpair2(add2(sums[0], sums[1]));
        const float sum = sum2.x + sum2.y;
        etc::tmem_wait_st();
        // A row that has seen nothing has no weights: its masked scores leave 2^-126 each in a quarter of the exponentials, and a
        // sum of those is not a sum to divide by.
        l = fmaf(sum, odd ? 0.f : exp2f(b - ev), l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(p_full(i));
      }
      // ---- results
      wait(pv_done(i), (tile - 1) & 1);
      tc_fence_after();
      const bool cut = s.t0 > 0 || s.t1 < s.nt;
      mine->x = l;
      named_sync(1 + i, 256);
      l += theirs->x;
      named_sync(1 + i, 256);
      if (!cut) {
        const float up = exp2f(0.5f * b), f = l > 0.f ? up / l : 0.f;   // in two steps: no overflow
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + oat + half * (D / 2));
#pragma unroll 1
        for (int q4 = 0; q4 < D / 64; ++q4) {
          uint32_t v[32];
          tmem_ld32(co, v, 32 * q4);
          tmem_wait_ld(v);
          if (live)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float y0 = __uint_as_float(v[8 * k + 2 * x]) * f * up, y1 = __uint_as_float(v[8 * k + 2 * x + 1]) * f * up;
                w[x] = a.q_dtype == TQ_F16 ? half2_bits(y0, y1) : etc::bf16x2_bits(y0, y1);
              }
              o[4 * q4 + k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
      } else {
        // slot 2 c: the item began before this CTA; 2 c + 1: it goes on behind it
        float4* part = reinterpret_cast<float4*>(a.p.part) + (int64_t)(2 * blockIdx.x + (s.t0 == 0 ? 1 : 0)) * (D / 4 + 1) * kItemRows;
#pragma unroll 1
        for (int q4 = 0; q4 < D / 64; ++q4) {
          uint32_t v[32];
          tmem_ld32(co, v, 32 * q4);
          tmem_wait_ld(v);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            part[(D / 8 * half + 8 * q4 + k) * kItemRows + 128 * i + r] =
                make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]), __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
        }
        if (half == 0) part[(D / 4) * kItemRows + 128 * i + r] = make_float4(m, l, b, 0.f);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(o_free(i));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u) : "memory");
}

// Grid: (CTAs of flash, D / 16): an item that begins in CTA c and goes on behind it; thread = row, 16 coordinates per CTA.
template <int D>
__global__ void __launch_bounds__(kItemRows) paged_flash_merge_kernel(FlashArgs a) {
  const int c = blockIdx.x, P = a.ctas, r = threadIdx.x;
  grid_dep_launch();
  grid_dep_wait();
  const int items = a.p.head[1], units = a.p.head[2];
  const int64_t U = (int64_t)units * a.heads;
  if (whole_items(a)) return;
  const Span sp = span_of(U, c, P);
  if (sp.u0 >= sp.u1) return;
  const Segment s = segment_at(a, items, units, sp.u1 - 1, sp.u1);
  if (s.first < sp.u0 || s.next <= sp.u1) return;   // began earlier, or ends here
  if (r >= s.nrows) return;
  const float4* part = reinterpret_cast<const float4*>(a.p.part);
  constexpr int kSlot = (D / 4 + 1) * kItemRows;
  float M = -INFINITY, unit = -INFINITY;   // the largest reference and the largest unit
  int slots = 0;
  for (int e = c; e < P; ++e) {
    const Span q = span_of(U, e, P);
    if (q.u0 >= s.next) break;
    const int t0 = max(0, (int)(max(q.u0, s.first) - s.first) - kItemCost), t1 = max(0, (int)(min(q.u1, s.next) - s.first) - kItemCost);
    if (t1 <= t0) continue;
    if (t0 == 0 && t1 == s.nt) return;   // one CTA had all of its tiles and wrote the result
    const float4 st = part[(int64_t)(2 * e + (t0 == 0 ? 1 : 0)) * kSlot + (D / 4) * kItemRows + r];
    if (st.x > M) unit += M == -INFINITY ? 0.f : M - st.x, M = st.x;   // relative to M
    unit = fmaxf(unit, st.x == -INFINITY ? -INFINITY : st.x - M + st.z);
    ++slots;
  }
  if (slots == 0) return;
  float acc[16], l = 0.f;
#pragma unroll
  for (int x = 0; x < 16; ++x) acc[x] = 0.f;
  for (int e = c; e < P; ++e) {
    const Span q = span_of(U, e, P);
    if (q.u0 >= s.next) break;
    const int t0 = max(0, (int)(max(q.u0, s.first) - s.first) - kItemCost), t1 = max(0, (int)(min(q.u1, s.next) - s.first) - kItemCost);
    if (t1 <= t0) continue;
    const float4* p = part + (int64_t)(2 * e + (t0 == 0 ? 1 : 0)) * kSlot;
    const float4 st = p[(D / 4) * kItemRows + r];
    const float w = st.x == -INFINITY ? 0.f : exp2f(st.x - M);
    l = fmaf(w, st.y, l);
    const float wv = st.x == -INFINITY || st.z == -INFINITY ? 0.f : exp2f((st.x - M + st.z) - unit);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = p[(4 * blockIdx.y + k) * kItemRows + r];
      acc[4 * k] = fmaf(wv, v.x, acc[4 * k]), acc[4 * k + 1] = fmaf(wv, v.y, acc[4 * k + 1]);
      acc[4 * k + 2] = fmaf(wv, v.z, acc[4 * k + 2]), acc[4 * k + 3] = fmaf(wv, v.w, acc[4 * k + 3]);
    }
  }
  const float up = exp2f(0.5f * unit), f = l > 0.f ? up / l : 0.f;
  const int row = s.row0 + r, tok = row / a.G, hq = (a.head0 + s.h) * a.G + row - tok * a.G;
  uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (((int64_t)a.bt.q_start[s.b] + tok) * a.Hq + hq) * D + 16 * blockIdx.y);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float y0 = acc[8 * k + 2 * x] * f * up, y1 = acc[8 * k + 2 * x + 1] * f * up;
      w[x] = a.q_dtype == TQ_F16 ? half2_bits(y0, y1) : etc::bf16x2_bits(y0, y1);
    }
    o[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace paged
}  // namespace tqk
