// Attention of a few query rows per sequence and KV head (single tokens, a few drafted ones) over paged caches: d = 64 or
// 128, 2- or 4-bit codes, with or without d signs.
//
// softmax(scale q k^T) v with both sides rotated: <q, k> = <Pi q, c[idx] norm> + sqrt(pi/2) / m rnorm <S q, 2 sigma - 1>, and
// the output's sums stay in the codes' domain until the merge maps them back with Pi^T and S^T. Up to eight query rows
// share a pass over the packed rows; more come in eights, each with its own pass.
//
// What has to be moved are the packed rows, so they go from the page to the tensor cores' registers with as few
// instructions as possible. Even so it is the instructions that bound it, about 510 per 16 tokens (mse4, d = 128): 32
// sequences of up to 16384 keys, 4 KV heads, take 73 us with issue slots 57 %, ALU 50 % and LSU 48 % busy, tensor pipe
// 15 %, where the bytes alone would take 25; 128 registers a thread leave 16 warps on an SM.
// A chunk is 16 tokens of one page (pages are multiples of 16): its codes, signs and norms are contiguous, and a warp
// streams its chunks through a ring of its own with 16-byte asynchronous copies. Scores are
// m16n8k16 products with the 16 tokens as rows and the query rows as columns: a lane's operand registers are pairs of
// coordinates of one token, which a table turns out of one packed byte (a copy of the table for each bank, so that no two
// lanes meet). Coordinates are numbered so that a lane's share of a token's row is contiguous. The value product has
// coordinates as rows and tokens as its inner dimension: two tokens' table entries, interleaved; its weights are the scores'
// registers, transposed across the warp (movmatrix). Weights carry the value norms, and each query row its own power of two
// that keeps its largest product of the two between 2^-13 and 2^12: norms of tokens that the row does not see, or hardly, cost
// it no digits. The sums stay in the codes' domain and the merge rotates them back.
//
// Work is cut evenly: CTA c of P takes units [c U / P, (c + 1) U / P) of the batch's U chunks (sequence by sequence, head by
// head), whatever the sequences' lengths; a CTA's part of one (sequence, head) is one partial result.
#pragma once

#include "paged_flash.cuh"

namespace tqk {
namespace paged {

constexpr int kDcWarps = 8, kDcThreads = 32 * kDcWarps;
constexpr int kDcMaxB = 2048;    // sequences whose running sums fit shared memory
constexpr int kChunk = 16;

template <int D, int BK, int BV, bool SG>
struct DcLayout {
  static constexpr int kRowK = D * BK / 8, kRowV = D * BV / 8, kRowS = SG ? D / 8 : 0;
  // one chunk: codes, signs, norms, residual norms of the keys, then of the values
  static constexpr int kSignK = kChunk * kRowK, kNormK = kSignK + kChunk * kRowS, kEndK = kNormK + (SG ? 64 : 32) * 2;
  static constexpr int kSignV = kEndK + kChunk * kRowV, kNormV = kSignV + kChunk * kRowS, kStage = kNormV + (SG ? 64 : 32) * 2;
  static constexpr int kDV = D + (SG ? D : 0);
  // Two CTAs per SM: two tables leave room for one stage less; a warp's ring also holds its sums at an item's end.
  static constexpr int kStages = BK != BV ? 3 : SG && D == 128 ? 5 : 4;
  static constexpr int kWarpRing = kStages * kStage;
  static_assert(kWarpRing >= 8 * kDV * 4, "a warp's sums must fit its ring");
  // The tables lie at a multiple of 32 KB of the shared window, so that a packed byte's offset and the lane's are or-ed
  // into the address; as many warps' rings as fit lie before them, the others, then the statistics behind.
  static constexpr int kTables = BK == BV ? 1 : 2;
  static constexpr int kFrontWarps = (32768 - 2048) / kWarpRing < kDcWarps ? (32768 - 2048) / kWarpRing : kDcWarps;
  static constexpr uint32_t kBack = kTables * 32768;                                    // from the tables on
  static constexpr uint32_t kStat = kBack + (kDcWarps - kFrontWarps) * kWarpRing;       // float [2][8 warps][8 rows]
  static constexpr uint32_t kPre = kStat + kDcWarps * 64;                               // int64 [B + 1]
  // dynamic shared memory for B sequences: the window begins at most 2 KB (static and reserved memory) in
  static constexpr size_t bytes(int B) { return 32768 + kPre + (size_t)(B + 1) * 8; }
};

struct DecodeArgs {
  AttnArgs a;
  int ctas;
};

__device__ __forceinline__ int small_tokens(const AttnArgs& a, int b) {
  const int n = seq_tokens(a.bt, b);
  return n > 0 && (int64_t)n * a.G <= a.small_rows ? n : 0;
}
// The query rows of one KV head come in eights. Each (KV head, eight) is a head of its own to the kernels here, a strip; a
// sequence has at most most_strips, which the grids and the workspace are made for.
__device__ __forceinline__ int eights(const AttnArgs& a, int n) { return (n * a.G + 7) >> 3; }
__device__ __forceinline__ int most_strips(const AttnArgs& a) { return a.Hkv * (a.small_rows >> 3); }
struct Strip {
  int h, row0, rows;   // KV head; its first query row (row = token * G + head within the group), their number
};
__device__ __forceinline__ Strip strip_of(const AttnArgs& a, int n, int hv) {
  const int e = eights(a, n), h = hv / e, row0 = 8 * (hv - h * e);
  return {h, row0, min(8, n * a.G - row0)};
}
// Query row `row` of KV head h among the rows of the call's q and out.
__device__ __forceinline__ int64_t row_of(const AttnArgs& a, int b, int h, int row) {
  const int i = row / a.G;
  return ((int64_t)a.bt.q_start[b] + i) * a.Hq + h * a.G + row - i * a.G;
}
// Chunks of one head of sequence b, and its first.
__device__ __forceinline__ int small_chunks(const AttnArgs& a, int b, int n, int& first) {
  first = 0;
  if (n == 0) return 0;
  int lo, hi;
  key_range(a.bt, b, 0, n - 1, n, a.causal, a.window, lo, hi);
  first = lo / kChunk;
  return hi > lo ? (hi + kChunk - 1) / kChunk - first : 0;
}

// Running sums over the sequences of chunks * strips into pre[0 .. B], by the whole CTA of NT threads; returns the most chunks
// of one (sequence, head).
template <int NT>
__device__ __forceinline__ int chunk_sums(const AttnArgs& a, int64_t* pre, int64_t* warp_s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t done = 0;
  int most = 0;
  for (int b0 = 0; b0 < a.bt.B; b0 += NT) {
    const int b = b0 + tid;
    int nch = 0, n = 0;
    if (b < a.bt.B) {
      int first;
      n = small_tokens(a, b);
      nch = small_chunks(a, b, n, first);
      if (blockIdx.x == 0 && seq_cut_short(a.bt, b)) report_error(a.err, kErrPaged);
    }
    const int64_t v = (int64_t)nch * (a.Hkv * eights(a, n));
    int64_t incl = v;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    const int top = __reduce_max_sync(0xffffffffu, nch);
    if (lane == 31) warp_s[warp] = incl, warp_s[NT / 32 + warp] = top;
    __syncthreads();
    int64_t before = done;
    for (int w = 0; w < warp; ++w) before += warp_s[w];
    if (b < a.bt.B) pre[b] = before + incl - v;
    for (int w = 0; w < NT / 32; ++w) done += warp_s[w], most = max(most, (int)warp_s[NT / 32 + w]);
    __syncthreads();
  }
  if (tid == 0) pre[a.bt.B] = done;
  __syncthreads();
  return most;
}

// How the units are shared out. While every (sequence, head) is short and has a CTA, each CTA takes one and finishes it: no
// partial results (up to 96 chunks, 12 for each warp: a call for 16 x 12 heads of 1200 keys takes 23 us so and 29 us cut).
// Otherwise evenly, with at least 8 chunks for a CTA, one for each warp.
constexpr int kWholeChunks = 96;
__device__ __forceinline__ bool take_whole(const AttnArgs& a, int most, int ctas) {
  return most <= kWholeChunks && (int64_t)a.bt.B * most_strips(a) <= ctas;
}
__device__ __forceinline__ int even_parts(int64_t U, int ctas) { return (int)min((int64_t)ctas, max((int64_t)1, U >> 3)); }

__device__ __forceinline__ int last_at_or_before64(const int64_t* start, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
// Byte offset of (token row r, byte o) among a chunk's rows of RB bytes: rows and 32-byte halves trade places so that the
// lanes of one access (tokens r, r + 4 together, or t + 4 j for t = 0 .. 3) fall into different banks.
template <int RB>
__device__ __forceinline__ int spot(int r, int o) {
  if (RB == 64) return ((r >> 1) << 7) + (((r & 1) ^ ((r >> 2) & 1)) << 6) + (o ^ (((r >> 1) & 1) << 5));
  if (RB == 32) return ((r >> 2) << 7) + (((r & 3) ^ (((r >> 2) & 1) << 1)) << 5) + o;
  return r * RB + o;
}
// N bytes (2, 4, 8 or 16) from shared memory as words.
template <int N>
__device__ __forceinline__ void lds_bytes(uint32_t a, uint32_t* w) {
  if (N == 16) {
    const uint4 v = lds128(a);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if (N == 8) {
    const uint2 v = lds64(a);
    w[0] = v.x, w[1] = v.y;
  } else if (N == 4) {
    w[0] = lds32(a);
  } else {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(a));
    w[0] = v;
  }
}
__device__ __forceinline__ float lds_half(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(a));
  return __half2float(__ushort_as_half(v));
}
// The pairs of coordinates in byte i of w: 4 bits one pair, 2 bits two (x: coordinates 0, 1; y: 2, 3).
// at4, at8: the lane's copy in the table's first row, at a multiple of 32 KB.
template <int B>
__device__ __forceinline__ uint2 lut_byte(uint32_t w, int i, uint32_t at4, uint32_t at8) {
  if (B == 4) return make_uint2(table32(byte128(w, i) | at4), 0);
  return table64(byte128(w, i) | at8);
}

// out[r][j] = sum_i in[r][i] T[i][j] for nr <= 8 rows (16-byte aligned) and a D x D matrix; a thread asks for all of its share of T at once (one
// latency where rows_matvec has four). part_s: [8][256] floats. Not inlined: its code is fetched once for up to four products.
template <int D>
__device__ __noinline__ void rows_at_once(const float* in, int nr, const float* T, float* part_s, float* out) {
  constexpr int kParts = kDcThreads / D, kShare = D / kParts;
  const int tid = threadIdx.x, j = tid % D, part = tid / D;
  float p[kShare];
#pragma unroll
  for (int i = 0; i < kShare; ++i) p[i] = __ldg(T + (size_t)(part * kShare + i) * D + j);
#pragma unroll 2
  for (int r = 0; r < nr; ++r) {
    const float4* x = reinterpret_cast<const float4*>(in + r * D + part * kShare);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kShare / 4; ++i) {
      const float4 v = x[i];
      acc[0] = fmaf(v.x, p[4 * i], acc[0]), acc[1] = fmaf(v.y, p[4 * i + 1], acc[1]);
      acc[2] = fmaf(v.z, p[4 * i + 2], acc[2]), acc[3] = fmaf(v.w, p[4 * i + 3], acc[3]);
    }
    part_s[(r * kParts + part) * D + j] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  }
  __syncthreads();
  for (int e = tid; e < nr * D; e += kDcThreads) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kParts; ++q) s += part_s[(e / D * kParts + q) * D + e % D];
    out[e] = s;
  }
  __syncthreads();
}

// ONE: the tables are so narrow that every item is whole; the CTA prepares its queries itself, and this is the call's only
// kernel.
template <int D, int BK, int BV, bool SG, bool NF16, bool ONE>
__global__ void __launch_bounds__(kDcThreads, 2) paged_decode_kernel(DecodeArgs da) {
  using L = DcLayout<D, BK, BV, SG>;
  extern __shared__ __align__(128) unsigned char smem_dc[];
  const AttnArgs& a = da.a;
  const uint32_t base = smem_addr(smem_dc), lut = (base + 32767u) & ~32767u;
  unsigned char* const tables = smem_dc + (lut - base);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  int64_t* pre = reinterpret_cast<int64_t*>(tables + L::kPre);
  float* stat = reinterpret_cast<float*>(tables + L::kStat);   // [warp][row] maximum, then [warp][row] sum
  __shared__ int64_t warp_s[2 * kDcWarps];
  if (lut - base < L::kFrontWarps * L::kWarpRing) {   // more static memory than expected
    if (tid == 0) report_error(a.err, kErrInternal);
    return;
  }
  grid_dep_launch();
  const int most = chunk_sums<kDcThreads>(a, pre, warp_s);
  const int64_t U = pre[a.bt.B];
  const bool whole = ONE || take_whole(a, most, gridDim.x);
  Span sp{0, 0};
  if (whole) {
    const int b = blockIdx.x / most_strips(a), hv = blockIdx.x - b * most_strips(a);
    const int n = b < a.bt.B ? small_tokens(a, b) : 0, strips = a.Hkv * eights(a, n);
    if (hv < strips) {
      const int64_t nch = (pre[b + 1] - pre[b]) / strips;
      sp = {pre[b] + hv * nch, pre[b] + (hv + 1) * nch};
      if (nch == 0) {   // no keys
        const Strip l = strip_of(a, n, hv);
        for (int e = tid; e < l.rows * D; e += kDcThreads)
          store_any(a.out, a.q_dtype, row_of(a, b, l.h, l.row0 + e / D) * D + e % D, 0.f);
      }
    }
  } else if ((int)blockIdx.x < even_parts(U, gridDim.x)) {
    sp = span_of(U, blockIdx.x, even_parts(U, gridDim.x));
  }
  if (sp.u0 >= sp.u1) {
    grid_dep_wait();   // every CTA waits: a kernel behind this one may count on the one before
    return;
  }
  const uint32_t k4 = lut | 4 * lane, k8 = lut | 8 * (lane & 15);
  const uint32_t v4 = k4 + (L::kTables - 1) * 32768, v8 = k8 + (L::kTables - 1) * 32768;
  const uint32_t ring_off = warp < L::kFrontWarps ? warp * L::kWarpRing : lut - base + L::kBack + (warp - L::kFrontWarps) * L::kWarpRing;
  const uint32_t ring = base + ring_off;
  constexpr int KB = L::kRowK / 4, VB = L::kRowV / 8;      // bytes of a row that a lane reads
  constexpr int KW = (KB + 3) / 4, VW = (VB + 3) / 4;
  // Two chunks are scored and weighted together (their products and table reads interleave) where the ring has room.
  constexpr int CN = L::kStages >= 4 && !SG ? 2 : 1;   // (with signs the registers do not do: 36 -> 40 us)
  constexpr int KS = D / 16;                               // inner steps of the score product, and row tiles of the value one
  const int tk = (g >> 1) + 4 * (g & 1);                   // the token of score row g (row g + 8: 8 later)
  bool tables_made = false;

  for (int64_t u = sp.u0; u < sp.u1;) {
    const int b = last_at_or_before64(pre, a.bt.B, u);
    const int n = small_tokens(a, b);
    int first;
    const int nch = small_chunks(a, b, n, first);
    const int hv = (int)((u - pre[b]) / nch);
    const int64_t item_u = pre[b] + (int64_t)hv * nch;
    const int c0 = (int)(u - item_u), c1 = (int)(min(sp.u1, item_u + nch) - item_u);
    u = item_u + nch;
    const Strip strip = strip_of(a, n, hv);
    const int h = strip.h, rows = strip.rows, len = a.bt.len[b];
    int lo_all, hi_all;
    key_range(a.bt, b, 0, n - 1, n, a.causal, a.window, lo_all, hi_all);
    // rows 2 t, 2 t + 1 are this lane's columns: the keys they see
    int lo[2], hi[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * t + j, pos = len - n + (strip.row0 + r) / a.G;
      lo[j] = 0, hi[j] = r < rows ? hi_all : 0;
      if (a.causal) {
        hi[j] = min(hi[j], pos + 1);
        if (a.window > 0) lo[j] = max(0, pos - a.window + 1);
      }
    }
    // ---- the warp's chunks: c0 + warp, + 8, ...; the ring holds those under way
    const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kDcWarps - 1) / kDcWarps : 0;
    unsigned there = 0;   // bit (i mod 32): chunk i lies on a valid page
    const uint32_t cpp = a.bt.page_size / kChunk;   // chunks of a page
    const uint32_t inv = cpp > 1 ? 0xffffffffu / cpp + 1u : 0u;   // exact below 2^26 chunks
    const int32_t* tab = a.bt.table + (int64_t)b * a.bt.max_pages;
    const uint32_t ch0 = first + c0 + warp;
    auto page_of = [&](int i) -> int {
      const uint32_t ch = ch0 + i * kDcWarps;
      return i < mine ? tab[cpp > 1 ? __umulhi(ch, inv) : ch] : -1;
    };
    // This lane's part in a copy: 16 bytes of the norms (lanes 0 ..), of the signs, and of each 512 bytes of codes.
    constexpr int NB = NF16 ? 2 : 4;   // bytes of a norm
    constexpr int NS = kChunk * L::kRowS / 16;
    const char* n_src = nullptr;
    uint32_t n_row = 0, n_dst = 0;
    if (lane < 2 * NB) {
      n_src = static_cast<const char*>(lane < NB ? a.kc.norms : a.vc.norms) + 16 * (lane & (NB - 1));
      n_row = kChunk * NB, n_dst = (lane < NB ? L::kNormK : L::kNormV) + 16 * (lane & (NB - 1));
    } else if (SG && lane < 2 * NB + 4) {
      const int x = lane - 2 * NB;
      n_src = reinterpret_cast<const char*>(x < 2 ? a.kc.rnorms : a.vc.rnorms) + 16 * (x & 1);
      n_row = 2 * kChunk, n_dst = (x < 2 ? L::kNormK : L::kNormV) + 64 + 16 * (x & 1);
    }
    const uint32_t k_dst = spot<L::kRowK>(lane / (L::kRowK / 16), lane % (L::kRowK / 16) * 16);
    const uint32_t v_dst = L::kEndK + spot<L::kRowV>(lane / (L::kRowV / 16), lane % (L::kRowV / 16) * 16);
    int page = -1;            // of the chunk that is fetched next
    uint32_t fill = 0;        // its stage's offset
    auto fetch = [&](int i) {
      bool ok = false;
      if (i < mine) {
        const uint32_t ch = ch0 + i * kDcWarps, pi = cpp > 1 ? __umulhi(ch, inv) : ch;
        ok = page >= 0 && page < a.bt.num_pages;
        if (ok) {
          const uint32_t at = ((uint32_t)page * a.Hkv + h) * cpp + (ch - pi * cpp);   // the chunk among all (below 2^32)
          const uint32_t st = ring + fill;
          const uint8_t* ck = a.kc.codes + (uint64_t)at * (kChunk * L::kRowK) + 16 * lane;
          const uint8_t* cv = a.vc.codes + (uint64_t)at * (kChunk * L::kRowV) + 16 * lane;
          // 32 lanes further is 8 rows (of 64 bytes) further, which the rows' places follow
          if (kChunk * L::kRowK / 16 >= 32 || lane < kChunk * L::kRowK / 16) cp16(st + k_dst, ck);
          if (kChunk * L::kRowK / 16 > 32) cp16(st + k_dst + 512, ck + 512);
          if (kChunk * L::kRowV / 16 >= 32 || lane < kChunk * L::kRowV / 16) cp16(st + v_dst, cv);
          if (kChunk * L::kRowV / 16 > 32) cp16(st + v_dst + 512, cv + 512);
          if (SG && lane < 2 * NS)
            cp16(st + (lane < NS ? L::kSignK + 16 * lane : L::kSignV + 16 * (lane - NS)),
                 (lane < NS ? a.kc.signs + 16 * lane : a.vc.signs + 16 * (lane - NS)) + (uint64_t)at * (kChunk * L::kRowS));
          if (n_src) cp16(st + n_dst, n_src + (uint64_t)at * n_row);
        } else if (lane == 0) {
          report_error(a.err, kErrPaged);
        }
        page = page_of(i + 1);
      }
      there = ok ? there | 1u << (i & 31) : there & ~(1u << (i & 31));
      fill = fill + L::kStage == L::kWarpRing ? 0 : fill + L::kStage;
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    page = page_of(0);
    for (int i = 0; i < L::kStages - CN; ++i) fetch(i);
    // ---- rotated queries, while the first copies are under way
    constexpr int DK = D + (SG ? D : 0);
    const float* src;
    if (ONE) {   // by this CTA, in the tables' place
      float* zf = reinterpret_cast<float*>(tables);     // [8][D]
      float* part_s = zf + 8 * D;                       // [8][256]
      float* o = part_s + 8 * 256;                      // [8][D]
      float* qq = o + 8 * D;                            // [8][DK]
      float z[D / 32], f1 = a.scale * 1.44269504089f;
      bool blind = false;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) z[c] = 0.f;
      if (warp < rows) {
        const int i = (strip.row0 + warp) / a.G;
        const int64_t t0 = a.bt.q_start[b] + i;
        const int64_t p = a.prep.pos ? (int64_t)a.prep.pos[t0] : (int64_t)len - n + i;
        if (a.prep.cos_sin && (p < 0 || p >= a.prep.max_pos)) {
          if (lane == 0 && (a.prep.pos || p >= 0)) report_error(a.err, kErrPaged);
          blind = true;   // it sees nothing
        } else {
          prep_head<float, D / 32>(a.q, a.q_dtype, t0 * a.q_stride + (int64_t)(h * a.G + strip.row0 + warp - i * a.G) * D, D, a.prep, p, z);
        }
      }
      f1 *= tame_head<D / 32>(z);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) zf[warp * D + lane + 32 * c] = z[c];
      __syncthreads();
      rows_at_once<D>(zf, rows, a.k.PiT, part_s, o);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) qq[warp * DK + lane + 32 * c] = blind ? kBlind : o[warp * D + lane + 32 * c] * f1;
      if (SG) {
        __syncthreads();
        rows_at_once<D>(zf, rows, a.k.ST, part_s, o);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) qq[warp * DK + D + lane + 32 * c] = blind ? kBlind : o[warp * D + lane + 32 * c] * (f1 * kQjlScale / (float)D);
      }
      __syncthreads();
      src = qq + g * DK;
    } else {
      if (!tables_made) {
        build_lut(a.k, tables, tid, kDcThreads);
        if (BK != BV) build_lut(a.v, tables + 32768, tid, kDcThreads);
      }
      grid_dep_wait();
      src = a.qr + (((int64_t)b * most_strips(a) + hv) * 8 + g) * DK;
    }
    // ---- queries: row g, this lane's coordinates, as f16 times a power of two
    uint32_t qc[2 * KS], qs[SG ? 2 * KS : 1];
    float fc[2], fs[2];
    {
      float z[D / 4];
      float top = 0.f;
      bool blind = false;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const float4 v = g < rows ? *reinterpret_cast<const float4*>(src + t * (D / 4) + 4 * x) : make_float4(0, 0, 0, 0);
        z[4 * x] = v.x, z[4 * x + 1] = v.y, z[4 * x + 2] = v.z, z[4 * x + 3] = v.w;
      }
      blind = is_blind(z[0]);
#pragma unroll
      for (int x = 0; x < D / 4; ++x) z[x] = blind ? 0.f : z[x];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (__shfl_sync(0xffffffffu, (int)blind, 8 * t + 4 * j)) hi[j] = 0;
#pragma unroll
      for (int x = 0; x < D / 4; ++x) top = fmaxf(top, fabsf(z[x]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = 0;
      if (top > 0.f && top < INFINITY) frexpf(top, &e);
      e = max(-126, min(126, e));   // 2^-e is a number too
      float dn = ldexpf(1.f, -e), upf = ldexpf(1.f, e);
#pragma unroll
      for (int s = 0; s < KS; ++s)
        qc[2 * s] = half2_bits(z[4 * s] * dn, z[4 * s + 1] * dn), qc[2 * s + 1] = half2_bits(z[4 * s + 2] * dn, z[4 * s + 3] * dn);
      upf /= a.k.cent_up;   // the tables' factor, out again
      fc[0] = __shfl_sync(0xffffffffu, upf, 8 * t), fc[1] = __shfl_sync(0xffffffffu, upf, 8 * t + 4);
      if (SG) {
        // this lane's signs are those of projections t D/4 .. : step s takes pairs (i, i + D/8), i = 2 s, 2 s + 1
        top = 0.f;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const float4 v = g < rows && !blind ? *reinterpret_cast<const float4*>(src + D + t * (D / 4) + 4 * x) : make_float4(0, 0, 0, 0);
          z[4 * x] = v.x, z[4 * x + 1] = v.y, z[4 * x + 2] = v.z, z[4 * x + 3] = v.w;
        }
#pragma unroll
        for (int x = 0; x < D / 4; ++x) top = fmaxf(top, fabsf(z[x]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        e = 0;
        if (top > 0.f && top < INFINITY) frexpf(top, &e);
        e = max(-126, min(126, e));
        dn = ldexpf(1.f, -e), upf = ldexpf(1.f, e);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qs[2 * s] = half2_bits(z[2 * s] * dn, z[2 * s + D / 8] * dn);
          qs[2 * s + 1] = half2_bits(z[2 * s + 1] * dn, z[2 * s + 1 + D / 8] * dn);
        }
        fs[0] = __shfl_sync(0xffffffffu, upf, 8 * t), fs[1] = __shfl_sync(0xffffffffu, upf, 8 * t + 4);
      }
    }
    if (!tables_made) {
      tables_made = true;
      if (ONE) {
        __syncthreads();   // the queries have been read
        build_lut(a.k, tables, tid, kDcThreads);
        if (BK != BV) build_lut(a.v, tables + 32768, tid, kDcThreads);
      }
      __syncthreads();
    }
    int lo_w = max(lo[0], lo[1]), hi_w = min(2 * t < rows ? hi[0] : INT_MAX, 2 * t + 1 < rows ? hi[1] : INT_MAX);
    lo_w = max(lo_w, __shfl_xor_sync(0xffffffffu, lo_w, 1)), lo_w = max(lo_w, __shfl_xor_sync(0xffffffffu, lo_w, 2));
    hi_w = min(hi_w, __shfl_xor_sync(0xffffffffu, hi_w, 1)), hi_w = min(hi_w, __shfl_xor_sync(0xffffffffu, hi_w, 2));
    float oc[KS][4], os[SG ? KS : 1][4];
#pragma unroll
    for (int x = 0; x < KS; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) oc[x][j] = 0.f;
#pragma unroll
    for (int x = 0; x < (SG ? KS : 1); ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) os[x][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float sv[2] = {0.f, 0.f};   // what weight times value norm is multiplied by, a power of two; 0: no value yet

    uint32_t use = 0;         // the offset of the stage in use
    auto next = [](uint32_t at) -> uint32_t { return at + L::kStage == L::kWarpRing ? 0 : at + L::kStage; };
    for (int i = 0; i < mine; i += CN) {
      __syncwarp();   // the stages that are filled next have been read by every lane
#pragma unroll
      for (int c = 0; c < CN; ++c) fetch(i + L::kStages - CN + c);
      asm volatile("cp.async.wait_group %0;\n" ::"n"(L::kStages - CN) : "memory");
      __syncwarp();
      uint32_t stage[CN];
#pragma unroll
      for (int c = 0; c < CN; ++c) stage[c] = ring + use, use = next(use);
      float xs[CN][4], vn[CN][2], wn[CN][2];   // scores, then weights; value norms; their signs' norms
#pragma unroll
      for (int c = 0; c < CN; ++c) {
        const uint32_t st = stage[c];
        const bool here = i + c < mine && (there >> ((i + c) & 31) & 1);
        const int key0 = (ch0 + (i + c) * kDcWarps) * kChunk;
        auto norm_at = [&](uint32_t off, int r) -> float {
          if (NF16) return lds_half(st + off + 2 * r);
          return __uint_as_float(lds32(st + off + 4 * r));
        };
        // ---- scores of tokens tk, tk + 8 (rows g, g + 8) for query rows 2 t, 2 t + 1
        float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        {
          uint32_t w0[KW], w1[KW];
          lds_bytes<KB>(st + spot<L::kRowK>(tk, KB * t), w0);
          lds_bytes<KB>(st + spot<L::kRowK>(tk + 8, KB * t), w1);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            uint32_t a0, a1, a2, a3;
            if (BK == 4) {
              a0 = lut_byte<4>(w0[s >> 1], 2 * (s & 1), k4, k8).x, a2 = lut_byte<4>(w0[s >> 1], 2 * (s & 1) + 1, k4, k8).x;
              a1 = lut_byte<4>(w1[s >> 1], 2 * (s & 1), k4, k8).x, a3 = lut_byte<4>(w1[s >> 1], 2 * (s & 1) + 1, k4, k8).x;
            } else {
              const uint2 x = lut_byte<2>(w0[s >> 2], s & 3, k4, k8), y = lut_byte<2>(w1[s >> 2], s & 3, k4, k8);
              a0 = x.x, a2 = x.y, a1 = y.x, a3 = y.y;
            }
            mma16816(s1, a0, a1, a2, a3, qc[2 * s], qc[2 * s + 1]);
          }
          if (SG) {
            uint32_t x, y;
            if (D == 128) {
              lds_bytes<4>(st + L::kSignK + tk * L::kRowS + 4 * t, &x);
              lds_bytes<4>(st + L::kSignK + (tk + 8) * L::kRowS + 4 * t, &y);
            } else {   // 16 signs: the upper eight to bits 16 .. 23
              lds_bytes<2>(st + L::kSignK + tk * L::kRowS + 2 * t, &x);
              lds_bytes<2>(st + L::kSignK + (tk + 8) * L::kRowS + 2 * t, &y);
              x = __byte_perm(x, 0, 0x4140), y = __byte_perm(y, 0, 0x4140);
            }
            x = ~x, y = ~y;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              auto two = [](uint32_t w, int k) { return ((w << (15 - k)) & 0x80008000u) ^ 0x3C003C00u; };
              mma16816(s2, two(x, 2 * s), two(y, 2 * s), two(x, 2 * s + 1), two(y, 2 * s + 1), qs[2 * s], qs[2 * s + 1]);
            }
          }
        }
        const float nA = norm_at(L::kNormK, tk), nB = norm_at(L::kNormK, tk + 8);
        float rA = 0.f, rB = 0.f;
        if (SG) rA = lds_half(st + L::kNormK + 64 + 2 * tk), rB = lds_half(st + L::kNormK + 64 + 2 * (tk + 8));
        float (&x)[4] = xs[c];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[j] = s1[j] * (nA * fc[j]);
          x[2 + j] = s1[2 + j] * (nB * fc[j]);
          if (SG) x[j] = fmaf(s2[j], rA * fs[j], x[j]), x[2 + j] = fmaf(s2[2 + j], rB * fs[j], x[2 + j]);
        }
        float vA = norm_at(L::kNormV, tk), vB = norm_at(L::kNormV, tk + 8), wA = 0.f, wB = 0.f;
        if (SG) wA = lds_half(st + L::kNormV + 64 + 2 * tk), wB = lds_half(st + L::kNormV + 64 + 2 * (tk + 8));
        if (!here || key0 < lo_w || key0 + kChunk > hi_w) {
          const int kA = key0 + tk, kB = kA + 8;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (!(here && kA >= lo[j] && kA < hi[j])) x[j] = -INFINITY;
            if (!(here && kB >= lo[j] && kB < hi[j])) x[2 + j] = -INFINITY;
          }
          // a token behind the sequence's end counts for nothing, whatever its slot holds
          if (!here || kA >= hi_all) vA = wA = 0.f;
          if (!here || kB >= hi_all) vB = wB = 0.f;
          // One that is not finite makes the rows that see it NaN by their scores: weight 0 times it would not be 0 for the others.
          const bool okA = fabsf(vA) + fabsf(wA) < INFINITY, okB = fabsf(vB) + fabsf(wB) < INFINITY;
          if (!okA || !okB) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (!okA && kA >= lo[j] && kA < hi[j]) x[j] = NAN;
              if (!okB && kB >= lo[j] && kB < hi[j]) x[2 + j] = NAN;
            }
            if (!okA) vA = wA = 0.f;
            if (!okB) vB = wB = 0.f;
          }
        }
        vn[c][0] = vA, vn[c][1] = vB, wn[c][0] = wA, wn[c][1] = wB;
      }
      float vt = fmaxf(vn[0][0], vn[0][1]), tops[2] = {fmaxf(xs[0][0], xs[0][2]), fmaxf(xs[0][1], xs[0][3])};
      if (CN == 2) {
        vt = fmaxf(vt, fmaxf(vn[CN - 1][0], vn[CN - 1][1]));
        tops[0] = fmaxf(tops[0], fmaxf(xs[CN - 1][0], xs[CN - 1][2])), tops[1] = fmaxf(tops[1], fmaxf(xs[CN - 1][1], xs[CN - 1][3]));
      }
      auto of_all = [](float x) -> float {   // the largest of a query row's eight lanes
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      };
      // Rarely: the reference of the weights moves, or the unit of the sums may have to (weights are below 2^8).
      if (__any_sync(0xffffffffu, tops[0] > m[0] + 8.f || tops[1] > m[1] + 8.f || vt * fmaxf(sv[0], sv[1]) > 16.f)) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float top = of_all(tops[j]), old = m[j];
          float back = 1.f;   // 2^(the old reference - the new)
          if (top > old) back = old == -INFINITY ? 0.f : ex2(old - top), m[j] = top;
          l[j] *= back;
          const float ref = m[j] == -INFINITY ? 0.f : m[j];
          float z = 0.f;
#pragma unroll
          for (int c = 0; c < CN; ++c)
            z = fmaxf(z, fmaxf(ex2(xs[c][j] - ref) * vn[c][0], ex2(xs[c][2 + j] - ref) * vn[c][1]));
          z = of_all(z);
          f[j] = 1.f;
          if (m[j] > old || z * sv[j] > 4096.f) {   // the largest product to about one
            int e = -100;
            if (z > 0.f && z < INFINITY) frexpf(z, &e);
            float now = z < INFINITY ? ldexpf(1.f, -max(-100, min(126, e))) : 0.f;
            if (sv[j] > 0.f) now = fminf(now, sv[j] * 1.1529215e18f);   // 2^60: the sums stay finite
            f[j] = sv[j] > 0.f ? now / sv[j] * back : 0.f, sv[j] = now;
          }
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int y = 0; y < KS; ++y) {
            oc[y][0] *= f[0], oc[y][1] *= f[1], oc[y][2] *= f[0], oc[y][3] *= f[1];
            if (SG) os[y][0] *= f[0], os[y][1] *= f[1], os[y][2] *= f[0], os[y][3] *= f[1];
          }
        }
      }
      const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
      for (int c = 0; c < CN; ++c) {
        float (&x)[4] = xs[c];
        const uint32_t st = stage[c];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[j] = ex2(x[j] - ref[j]), x[2 + j] = ex2(x[2 + j] - ref[j]);
          l[j] += x[j] + x[2 + j];
          x[j] *= sv[j], x[2 + j] *= sv[j];
        }
        const float vA = vn[c][0], vB = vn[c][1];
        const uint32_t b0 = movmatrix(half2_bits(x[0] * vA, x[1] * vA)), b1 = movmatrix(half2_bits(x[2] * vB, x[3] * vB));
        // ---- values: lane (g, t) holds coordinates g D/8 .. of tokens t, t + 4, t + 8, t + 12
        {
          uint32_t w[4][VW];
#pragma unroll
          for (int j = 0; j < 4; ++j) lds_bytes<VB>(st + L::kEndK + spot<L::kRowV>(t + 4 * j, VB * g), w[j]);
          if (BV == 4) {
            // The low nibbles of two tokens' bytes side by side, then the high ones: one table entry is the same coordinate
            // of both tokens (byte y: coordinate 2 y -> row g of tile y, 2 y + 1 -> row g + 8).
            uint32_t p[2][VW], q[2][VW];
#pragma unroll
            for (int x = 0; x < VW; ++x)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t wa = w[2 * j][x], wb = w[2 * j + 1][x];
                p[j][x] = (wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u);
                q[j][x] = ((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u);
              }
#pragma unroll
            for (int y = 0; y < KS; ++y)
              mma16816(oc[y], lut_byte<4>(p[0][y >> 2], y & 3, v4, v8).x, lut_byte<4>(q[0][y >> 2], y & 3, v4, v8).x,
                       lut_byte<4>(p[1][y >> 2], y & 3, v4, v8).x, lut_byte<4>(q[1][y >> 2], y & 3, v4, v8).x, b0, b1);
          } else {
#pragma unroll
            for (int y = 0; y < KS / 2; ++y) {   // byte y: coordinates 4 y .. 4 y + 3 -> tiles 2 y, 2 y + 1
              uint2 v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = lut_byte<2>(w[j][y >> 2], y & 3, v4, v8);
              mma16816(oc[2 * y], __byte_perm(v[0].x, v[1].x, 0x5410), __byte_perm(v[0].x, v[1].x, 0x7632),
                       __byte_perm(v[2].x, v[3].x, 0x5410), __byte_perm(v[2].x, v[3].x, 0x7632), b0, b1);
              mma16816(oc[2 * y + 1], __byte_perm(v[0].y, v[1].y, 0x5410), __byte_perm(v[0].y, v[1].y, 0x7632),
                       __byte_perm(v[2].y, v[3].y, 0x5410), __byte_perm(v[2].y, v[3].y, 0x7632), b0, b1);
            }
          }
          if (SG) {   // lane (g, t): signs of projections g D/8 .. of its four tokens; two tokens in one word
            const float wA = wn[c][0], wB = wn[c][1];
            const uint32_t r0 = movmatrix(half2_bits(x[0] * wA, x[1] * wA)), r1 = movmatrix(half2_bits(x[2] * wB, x[3] * wB));
            uint32_t sg[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (D == 128) {
                lds_bytes<2>(st + L::kSignV + (t + 4 * j) * L::kRowS + 2 * g, &sg[j]);
              } else {
                uint32_t v;
                asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(st + L::kSignV + (t + 4 * j) * L::kRowS + g));
                sg[j] = v;
              }
            }
            const uint32_t p = ~__byte_perm(sg[0], sg[1], 0x5410), q = ~__byte_perm(sg[2], sg[3], 0x5410);
#pragma unroll
            for (int y = 0; y < KS; ++y) {
              auto two = [](uint32_t w2, int k) { return ((w2 << (15 - k)) & 0x80008000u) ^ 0x3C003C00u; };
              mma16816(os[y], two(p, 2 * y), two(p, 2 * y + 1), two(q, 2 * y), two(q, 2 * y + 1), r0, r1);
            }
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    // ---- the warps' results, merged in their order
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
    }
    if (g == 0) {
      stat[warp * 8 + 2 * t] = m[0], stat[warp * 8 + 2 * t + 1] = m[1];
      stat[64 + warp * 8 + 2 * t] = l[0], stat[64 + warp * 8 + 2 * t + 1] = l[1];
    }
    __syncthreads();   // every warp is done with the ring
    float top[2];
    {
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        top[j] = -INFINITY;
        for (int w = 0; w < kDcWarps; ++w) top[j] = fmaxf(top[j], stat[w * 8 + 2 * t + j]);
        f[j] = m[j] == -INFINITY || sv[j] == 0.f ? 0.f : ex2(m[j] - top[j]) / sv[j];
      }
      const float fv[2] = {f[0] / a.v.cent_up, f[1] / a.v.cent_up};
      // sums [warp][coordinate][row]
      float* o = reinterpret_cast<float*>(smem_dc + ring_off);
#pragma unroll
      for (int y = 0; y < KS; ++y) {
        const int c = g * (D / 8) + 2 * y;
        *reinterpret_cast<float2*>(o + c * 8 + 2 * t) = make_float2(oc[y][0] * fv[0], oc[y][1] * fv[1]);
        *reinterpret_cast<float2*>(o + (c + 1) * 8 + 2 * t) = make_float2(oc[y][2] * fv[0], oc[y][3] * fv[1]);
        if (SG) {
          *reinterpret_cast<float2*>(o + (D + c) * 8 + 2 * t) = make_float2(os[y][0] * f[0], os[y][1] * f[1]);
          *reinterpret_cast<float2*>(o + (D + c + 1) * 8 + 2 * t) = make_float2(os[y][2] * f[0], os[y][3] * f[1]);
        }
      }
    }
    __syncthreads();
    float sum[L::kDV / 32];   // elements tid, tid + 256, ... of [coordinate][row]
#pragma unroll
    for (int k = 0; k < L::kDV / 32; ++k) {
      sum[k] = 0.f;
#pragma unroll
      for (int w = 0; w < kDcWarps; ++w)
        sum[k] += reinterpret_cast<const float*>(w < L::kFrontWarps ? smem_dc + w * L::kWarpRing
                                                                    : tables + L::kBack + (w - L::kFrontWarps) * L::kWarpRing)[tid + 256 * k];
    }
    float mt = -INFINITY, lt = 0.f;   // of row tid mod 8
    for (int w = 0; w < kDcWarps; ++w) mt = fmaxf(mt, stat[w * 8 + (tid & 7)]);
    for (int w = 0; w < kDcWarps; ++w) {
      const float mw = stat[w * 8 + (tid & 7)];
      lt += mw == -INFINITY ? 0.f : stat[64 + w * 8 + (tid & 7)] * ex2(mw - mt);
    }
    if (!whole) {
      float* part = a.part + ((int64_t)blockIdx.x + (int64_t)b * most_strips(a) + hv) * 8 * (L::kDV + 2);
#pragma unroll
      for (int k = 0; k < L::kDV / 32; ++k) part[tid + 256 * k] = sum[k];
      if (tid < 8) part[8 * L::kDV + tid] = mt, part[8 * L::kDV + 8 + tid] = lt;
      __syncthreads();   // before the ring and the statistics are written again
      continue;
    }
    // the only item: its result, through the first warps' rings
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem_dc);          // [8][D], then [8][D] of the signs
    float* part_s = acc + 8 * L::kDV;                        // [8][256]
    float* o1 = part_s + 8 * 256;                            // [8][D]
    static_assert((8 * L::kDV + 2048 + 8 * D) * 4 <= L::kFrontWarps * L::kWarpRing, "the finish must fit before the tables");
    const float inv_l = lt > 0.f ? 1.f / lt : 0.f;
#pragma unroll
    for (int k = 0; k < L::kDV / 32; ++k) {
      const int e = tid + 256 * k, r = e & 7, j = e >> 3;
      acc[j < D ? r * D + j : 8 * D + r * D + j - D] = sum[k] * inv_l;
    }
    __syncthreads();
    rows_at_once<D>(acc, rows, a.v.Pi, part_s, o1);
    float y[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) y[k] = o1[tid + 256 * k];
    if (SG) {
      __syncthreads();
      rows_at_once<D>(acc + 8 * D, rows, a.v.S, part_s, o1);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) y[k] = fmaf(kQjlScale / (float)D, o1[tid + 256 * k], y[k]);
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const int e = tid + 256 * k, r = e / D, x = e % D;
      if (r < rows) store_any(a.out, a.q_dtype, row_of(a, b, h, strip.row0 + r) * D + x, y[k]);
    }
  }
}

// ---- the small products around it: 8 rows times 32 columns of a constant matrix per CTA

// out[r][0 .. 31] = sum_i in[r][i] T[i][col .. col + 31] (row length ld) for 8 rows and ni <= 128: warp w sums its eighth of
// i; the eight parts meet in part_s ([8 warps][8 rows][32]) in a fixed order. The matrix's share is asked for at once, by
// the queries' kernel while its vectors are on their way (10 -> 8 us); the merge asks when its sums are made (asked before
// they are read, the registers cost those reads their overlap: 22 -> 31 us).
struct Slice {
  float p[16];
};
__device__ __forceinline__ Slice slice_of(const float* T, int ni, int ld, int col) {
  Slice s;
  const int share = ni / 8;
  const float* t = T + (size_t)((threadIdx.x >> 5) * share) * ld + col + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < 16; ++i) s.p[i] = i < share ? __ldg(t + (size_t)i * ld) : 0.f;
  return s;
}
__device__ __forceinline__ void rows_slice(const float* in, int ni, const Slice& T, float* part_s, float* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, share = ni / 8;   // ni: a multiple of 32
  float acc[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) acc[r] = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < share) {
#pragma unroll
      for (int r = 0; r < 8; ++r) acc[r] = fmaf(in[r * ni + warp * share + i], T.p[i], acc[r]);
    }
#pragma unroll
  for (int r = 0; r < 8; ++r) part_s[(warp * 8 + r) * 32 + lane] = acc[r];
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += part_s[w * 256 + tid];
  out[tid] = s;   // [8][32]
  __syncthreads();
}

// Queries of the small sequences, to qr [B][most strips][8][d + m]. Grid: (B * most strips, (d + m) / 32 column slices); 256
// threads: warp r prepares query row r of the strip.
__global__ void __launch_bounds__(256) paged_qslice_kernel(DecodeArgs da) {
  __shared__ float zf[8 * 128], part_s[8 * 256], ys[256];
  const AttnArgs& a = da.a;
  const int d = a.k.d, m = a.k.m, dk = d + m, tid = threadIdx.x, lane = tid & 31, r = tid >> 5;
  grid_dep_launch();
  const int b = blockIdx.x / most_strips(a), hv = blockIdx.x - b * most_strips(a);
  const int n = small_tokens(a, b);
  if (hv >= a.Hkv * eights(a, n)) return;
  const Strip l = strip_of(a, n, hv);
  const int col = 32 * blockIdx.y;
  const bool code = col < d;
  const Slice T = slice_of(code ? a.k.PiT : a.k.ST, d, code ? d : m, code ? col : col - d);
  float z[4] = {0.f, 0.f, 0.f, 0.f};
  bool blind = false;
  if (r < l.rows) {
    const int i = (l.row0 + r) / a.G;
    const int64_t t = a.bt.q_start[b] + i;
    const int64_t p = a.prep.pos ? (int64_t)a.prep.pos[t] : (int64_t)a.bt.len[b] - n + i;
    if (a.prep.cos_sin && (p < 0 || p >= a.prep.max_pos)) {
      if (lane == 0 && (a.prep.pos || p >= 0)) report_error(a.err, kErrPaged);
      blind = true;   // it sees nothing
    } else {
      prep_head<float, 4>(a.q, a.q_dtype, t * a.q_stride + (int64_t)(l.h * a.G + l.row0 + r - i * a.G) * d, d, a.prep, p, z);
    }
  }
  const float back = tame_head<4>(z);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < d) zf[r * d + lane + 32 * c] = z[c];
  __syncthreads();
  rows_slice(zf, d, T, part_s, ys);
  const float f = a.scale * 1.44269504089f * back * (code ? 1.f : kQjlScale / (float)m);
  a.qr[((int64_t)blockIdx.x * 8 + r) * dk + col + lane] = blind ? kBlind : ys[tid] * f;
}

// Grid: (B, most strips, d / 32): 32 coordinates of the rows of one (sequence, strip): its CTAs' parts merged in order, then
// o = (Pi_V^T acc + c S_V^T acc_s) / sum.
__global__ void __launch_bounds__(256) paged_decode_merge_kernel(DecodeArgs da) {
  extern __shared__ __align__(16) unsigned char smem[];
  const AttnArgs& a = da.a;
  const int d = a.v.d, m = a.v.m, dv = d + m, b = blockIdx.x, hv = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_launch();
  float* acc = reinterpret_cast<float*>(smem);        // [8][d], then [8][m]
  float* part_s = acc + 8 * dv;                       // [8][256]
  float* o1 = part_s + 8 * 256;                       // [256]
  float* o2 = o1 + 256;
  float* wgt = o2 + 256;                              // [CTAs][8] weights of the parts
  int* cta = reinterpret_cast<int*>(wgt + 8 * da.ctas);   // [CTAs] those that hold one
  __shared__ int64_t sums[8], sums2[8];
  __shared__ float f[8];
  __shared__ int parts, tops[8];
  const int n = small_tokens(a, b);
  if (hv >= a.Hkv * eights(a, n)) {
    grid_dep_wait();
    return;
  }
  int first;
  const int nch = small_chunks(a, b, n, first);
  // the units before this sequence, and all of them
  int64_t before = 0, all = 0;
  int most = 0;
  for (int x = tid; x < a.bt.B; x += 256) {
    int f0;
    const int tx = small_tokens(a, x), nx = small_chunks(a, x, tx, f0);
    const int64_t v = (int64_t)nx * (a.Hkv * eights(a, tx));
    most = max(most, nx);
    all += v;
    if (x < b) before += v;
  }
  for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o), all += __shfl_xor_sync(0xffffffffu, all, o);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) sums[warp] = before, sums2[warp] = all, tops[warp] = most;
  if (tid == 0) parts = 0;
  __syncthreads();
  before = all = 0;
  for (int w = 0; w < 8; ++w) before += sums[w], all += sums2[w], most = max(most, tops[w]);
  if (take_whole(a, most, da.ctas)) {   // finished already
    grid_dep_wait();
    return;
  }
  const int P = even_parts(all, da.ctas);
  const int64_t u0 = before + (int64_t)hv * nch, u1 = u0 + nch;
  if (warp == 0) {   // the CTAs whose units meet [u0, u1), in order; none if it is empty, though it may lie inside one's share
    int np = 0;
    for (int c0 = 0; c0 < P && nch > 0; c0 += 32) {
      const Span q = span_of(all, c0 + lane, P);
      const bool in = c0 + lane < P && q.u0 < q.u1 && q.u0 < u1 && q.u1 > u0;
      const unsigned who = __ballot_sync(0xffffffffu, in);
      if (in) cta[np + __popc(who & ((1u << lane) - 1))] = c0 + lane;
      np += __popc(who);
    }
    if (lane == 0) parts = np;
  }
  grid_dep_wait();
  __syncthreads();
  const int np = parts;
  const int64_t size = 8 * (int64_t)(dv + 2);
  const float* part = a.part + ((int64_t)b * most_strips(a) + hv) * size;
  {   // warp r: the weights of row r
    float top = -INFINITY, sum = 0.f;
    float mine = -INFINITY, part_sum = 0.f;   // of part `lane`; the others are read twice
    if (lane < np) {
      const float* p = part + cta[lane] * size + 8 * dv;
      mine = p[warp], part_sum = p[8 + warp];
    }
    top = mine;
    for (int c = lane + 32; c < np; c += 32) top = fmaxf(top, part[cta[c] * size + 8 * dv + warp]);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int c = lane; c < np; c += 32) {
      if (c >= 32) {
        const float* p = part + cta[c] * size + 8 * dv;
        mine = p[warp], part_sum = p[8 + warp];
      }
      const float w = mine == -INFINITY ? 0.f : ex2(mine - top);
      wgt[c * 8 + warp] = w;
      sum = fmaf(w, part_sum, sum);
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) f[warp] = sum > 0.f ? 1.f / sum : 0.f;
  }
  __syncthreads();
  const int col = 32 * blockIdx.z;
  {   // thread: elements tid, tid + 256, ... of the sums, all of row tid mod 8
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
    const int nk = dv / 32;
#pragma unroll 8
    for (int c = 0; c < np; ++c) {
      const float w = wgt[c * 8 + (tid & 7)];
      const float* p = part + cta[c] * size + tid;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < nk) v[k] = fmaf(w, p[256 * k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = tid + 256 * k, r = e & 7, j = e >> 3;
      if (k < nk) acc[j < d ? r * d + j : 8 * d + r * m + j - d] = v[k];
    }
  }
  const Slice tc = slice_of(a.v.Pi, d, d, col);
  Slice ts;
  if (m > 0) ts = slice_of(a.v.S, m, d, col);
  __syncthreads();
  rows_slice(acc, d, tc, part_s, o1);
  if (m > 0) rows_slice(acc + 8 * d, m, ts, part_s, o2);
  const Strip l = strip_of(a, n, hv);
  if (warp >= l.rows) return;
  float v = o1[tid];
  if (m > 0) v = fmaf(kQjlScale / (float)m, o2[tid], v);
  store_any(a.out, a.q_dtype, row_of(a, b, l.h, l.row0 + warp) * d + col + lane, v * f[warp]);
}

}  // namespace paged
}  // namespace tqk
