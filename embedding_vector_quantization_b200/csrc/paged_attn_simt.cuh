// Attention of a ragged batch over paged caches, any format (d <= 256, m <= 256, any query type): the general kernels.
//
// Query rows (token, head) are prepared and rotated into the domain of the codes, q' = scale log2(e) [Pi_K z ; c S_K z]
// with c = sqrt(pi/2) / m, so a key's score is |k| <q'_1, c[idx]> + rnorm <q'_2, 2 sigma - 1> in units of log2; a CTA takes
// 8 rows of one KV head and walks a split of their keys with a running maximum and sum; the combine merges the splits
// and maps the value sums back, o = (Pi_V^T acc + c S_V^T acc_s) / sum p ("TurboQuant / PolarQuant / QJL technical deep
// dive" (gemilab.net), "Scaled dot-product attention"). All of it in fp32.
//
// Bound by fp32 arithmetic: an element of a row is decoded once for 8 query rows and costs each a product. One token for
// each of 32 sequences of up to 16384 keys, 4 KV heads: 1.1 ms, 0.09 on the tensor cores; four prompts of up to 4096
// tokens: 35 ms, 0.38.
#pragma once

#include "paged_append.cuh"

namespace tqk {
namespace paged {

constexpr int kTileRows = 8;
constexpr int kKeyTile = 32;
constexpr int kAttThreads = 128;

struct AttnArgs {
  const void* q;
  int64_t q_stride;
  int q_dtype, Hq, Hkv, G;
  Batch bt;
  Prep prep;
  Quant k, v;
  CacheView kc, vc;
  float scale;
  int causal, window, nsplit;
  int small_rows;  // the single-token kernels: sequences with at most this many query rows
  float* qr;       // [ntok * Hq][dk] rotated queries (general kernels)
  float* part;     // partial results
  void* out;
  int* err;
};

// Tile `tile` of the batch: sequence, first row (row = token within the sequence * G + head within the group) and row count.
struct Tile {
  int b, row0, nrows;
};

// Every lane of the calling warp gets the tile (b = -1: past the last). Tiles are numbered sequence by sequence.
__device__ __forceinline__ Tile warp_find_tile(const Batch& bt, int G, int tile_rows, int tile) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b0 = 0; b0 < bt.B; b0 += 32) {
    const int b = b0 + lane;
    const int n = b < bt.B ? seq_tokens(bt, b) : 0;
    const int nt = (n * G + tile_rows - 1) / tile_rows;
    int incl = nt;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const bool mine = tile >= before + incl - nt && tile < before + incl;
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    if (who) {
      const int src = __ffs(who) - 1;
      Tile t;
      t.b = b0 + src;
      const int first = __shfl_sync(0xffffffffu, before + incl - nt, src);
      const int rows = __shfl_sync(0xffffffffu, n, src) * G;
      t.row0 = (tile - first) * tile_rows;
      t.nrows = min(tile_rows, rows - t.row0);
      return t;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return {-1, 0, 0};
}

// Keys [lo, hi) that some row of tokens i0 .. i1 (of n) of sequence b sees.
__device__ __forceinline__ void key_range(const Batch& bt, int b, int i0, int i1, int n, int causal, int window, int& lo, int& hi) {
  const int len = max(0, bt.len[b]);
  const int cap = (int)min((int64_t)len, (int64_t)bt.max_pages * bt.page_size);
  lo = 0, hi = cap;
  if (!causal) return;
  hi = min(cap, len - n + i1 + 1);
  if (window > 0) lo = max(0, len - n + i0 - window + 1);
  hi = max(hi, lo);
}

// What the rotated query of a row holds that sees nothing, because its rotation position is out of range: one bit pattern
// of NaN (a NaN of a computed query is another).
#define TQ_BLIND_BITS 0x7fb1b1b1
#define kBlind __int_as_float(TQ_BLIND_BITS)
__device__ __forceinline__ bool is_blind(float x) { return __float_as_int(x) == TQ_BLIND_BITS; }

__host__ __device__ inline size_t qprep_smem_bytes(int d, int m, int R) {
  const int w = d > m ? d : m;
  return (size_t)R * d * 4 + (size_t)R * w * 4 + (size_t)kAppThreads * R * 4;
}

// Grid: ceil(ntok * Hq / R). Rows of padding get q' = 0, rows whose rotation position is out of range kBlind.
template <int R>
__global__ void __launch_bounds__(kAppThreads) paged_qprep_kernel(AttnArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int d = a.k.d, m = a.k.m, dk = d + m, w = max(d, m);
  float* zf = reinterpret_cast<float*>(smem);
  float* ys = zf + (size_t)R * d;
  float* part_s = ys + (size_t)R * w;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int blind[R];
  __shared__ float back[R];   // of tame_head
  const int64_t row0 = (int64_t)blockIdx.x * R, rows = a.bt.ntok * a.Hq;
  if (tid < R) blind[tid] = 0;
  __syncthreads();
  for (int r = warp; r < R; r += kAppThreads / 32) {
    const int64_t row = row0 + r, t = row / a.Hq;
    const int h = (int)(row - t * a.Hq);
    const int b = row < rows ? warp_find_seq(a.bt, t) : -1;
    float z[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) z[c] = 0.f;
    if (b >= 0) {
      const int64_t p = a.prep.pos ? (int64_t)a.prep.pos[t] : (int64_t)a.bt.len[b] - a.bt.q_start[b + 1] + t;
      if (a.prep.cos_sin && (p < 0 || p >= a.prep.max_pos)) {
        // (a negative position of its own needs no report: the row sees nothing)
        if (lane == 0 && (a.prep.pos || p >= 0)) report_error(a.err, kErrPaged);
        if (lane == 0) blind[r] = 1;
      } else {
        prep_head<float, 8>(a.q, a.q_dtype, t * a.q_stride + (int64_t)h * d, d, a.prep, p, z);
      }
    }
    const float f = tame_head<8>(z);
    if (lane == 0) back[r] = f;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (lane + 32 * c < d) zf[r * d + lane + 32 * c] = z[c];
  }
  __syncthreads();
  const float s1 = a.scale * 1.44269504089f, s2 = m > 0 ? s1 * kQjlScale / (float)m : 0.f;
  rows_matvec<R>(zf, d, a.k.PiT, d, part_s, ys);
  for (int e = tid; e < R * d; e += kAppThreads) {
    const int r = e / d;
    if (row0 + r < rows) a.qr[(row0 + r) * dk + (e - r * d)] = blind[r] ? kBlind : ys[e] * (s1 * back[r]);
  }
  if (m == 0) return;
  __syncthreads();
  rows_matvec<R>(zf, d, a.k.ST, m, part_s, ys);
  for (int e = tid; e < R * m; e += kAppThreads) {
    const int r = e / m;
    if (row0 + r < rows) a.qr[(row0 + r) * dk + d + (e - r * m)] = ys[e] * (s2 * back[r]);
  }
}

// Expands the packed rows of `nt` tokens (their cache rows in at[], -1: not there) to fp32 rows of stride ld: norm c[idx],
// then rnorm (2 sigma - 1).
__device__ __forceinline__ void expand_rows(const Quant& Q, const CacheView& c, const int64_t* at, const float* cf, float* dst,
                                            int ld) {
  const int d = Q.d, m = Q.m, wd = (d + m) / 32;   // 32 coordinates at a time
  for (int e = threadIdx.x; e < kKeyTile * wd; e += kAttThreads) {
    const int t = e / wd, u = e - t * wd;
    const int64_t row = at[t];
    float* o = dst + t * ld + 32 * u;
    if (row < 0) {
      for (int i = 0; i < 32; ++i) o[i] = 0.f;
      continue;
    }
    const float n = load_norm(c.norms, Q.norm_dtype, row);
    if (32 * u < d) {
      if (Q.bits == 0) {
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
      } else {
        const uint32_t* words = reinterpret_cast<const uint32_t*>(c.codes + row * Q.codes_B);
        for (int i = 0; i < 32; ++i) o[i] = n * cf[packed_field(words, 32 * u + i, Q.bits)];
      }
    } else {
      const float w = Q.bits == 0 ? n : __half2float(c.rnorms[row]);
      const uint32_t s = reinterpret_cast<const uint32_t*>(c.signs + row * Q.signs_B)[u - d / 32];
      for (int i = 0; i < 32; ++i) o[i] = (s >> i) & 1 ? w : -w;
    }
  }
}

__host__ __device__ inline size_t attn_simt_smem_bytes(int dk, int dv) {
  const int w = dk > dv ? dk : dv;
  return (size_t)kTileRows * dk * 4 + (size_t)kKeyTile * (w + 1) * 4 + (size_t)kTileRows * kKeyTile * 4;
}

// Grid: (tiles, Hkv, nsplit). part: [tile][Hkv][nsplit][8 rows][dv + 2]: value sums, maximum, sum of weights.
__global__ void __launch_bounds__(kAttThreads) paged_attn_simt_kernel(AttnArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int dk = a.k.d + a.k.m, dv = a.v.d + a.v.m, ld = max(dk, dv) + 1;
  float* qs = reinterpret_cast<float*>(smem);                 // [8][dk]
  float* kv = qs + kTileRows * dk;                            // [32][ld]
  float* sc = kv + kKeyTile * ld;                             // [8][32]
  __shared__ int64_t at_k[kKeyTile], at_v[kKeyTile];
  __shared__ float ck[16], cv[16], mx[kTileRows], sm[kTileRows], al[kTileRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hk = blockIdx.y, split = blockIdx.z;
  if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0)
    for (int b = tid; b < a.bt.B; b += kAttThreads)
      if (seq_cut_short(a.bt, b)) report_error(a.err, kErrPaged);
  const Tile tl = warp_find_tile(a.bt, a.G, kTileRows, blockIdx.x);
  if (tl.b < 0) return;
  const int b = tl.b, tok0 = a.bt.q_start[b], n = a.bt.q_start[b + 1] - tok0;
  const int i0 = tl.row0 / a.G, i1 = (tl.row0 + tl.nrows - 1) / a.G;
  int lo, hi;
  key_range(a.bt, b, i0, i1, n, a.causal, a.window, lo, hi);
  const int span = ((hi - lo + a.nsplit - 1) / a.nsplit + kKeyTile - 1) / kKeyTile * kKeyTile;
  const int k0 = min(hi, lo + split * span), k1 = min(hi, k0 + span);
  const int pos_first = a.bt.len[b] - n;   // position of the sequence's first new token
  if (tid < 16) ck[tid] = (float)a.k.cent64()[tid], cv[tid] = (float)a.v.cent64()[tid];
  for (int e = tid; e < kTileRows * dk; e += kAttThreads) {
    const int r = e / dk, row = tl.row0 + r;
    float v = 0.f;
    if (r < tl.nrows) v = a.qr[((int64_t)(tok0 + row / a.G) * a.Hq + hk * a.G + row % a.G) * dk + (e - r * dk)];
    qs[e] = v;
  }
  if (tid < kTileRows) mx[tid] = -INFINITY, sm[tid] = 0.f;
  constexpr int kMaxAcc = (256 + 256) * kTileRows / kAttThreads;   // dv <= 512: columns tid, tid + 128, ... of 8 rows
  float acc[kMaxAcc];
#pragma unroll
  for (int i = 0; i < kMaxAcc; ++i) acc[i] = 0.f;

  for (int t0 = k0; t0 < k1; t0 += kKeyTile) {
    __syncthreads();
    if (tid < kKeyTile) {
      const int64_t at = t0 + tid < k1 ? place_of(a.bt, b, t0 + tid, hk, a.Hkv) : -1;
      if (at < 0 && t0 + tid < k1) report_error(a.err, kErrPaged);
      at_k[tid] = at, at_v[tid] = at;
    }
    __syncthreads();
    expand_rows(a.k, a.kc, at_k, ck, kv, ld);
    __syncthreads();
    for (int e = tid; e < kTileRows * kKeyTile; e += kAttThreads) {
      const int r = e / kKeyTile, t = e - r * kKeyTile;
      float s = 0.f;
      for (int i = 0; i < dk; ++i) s = fmaf(qs[r * dk + i], kv[t * ld + i], s);
      const int row = tl.row0 + r, p = pos_first + row / a.G, key = t0 + t;
      bool seen = r < tl.nrows && at_k[t] >= 0 && !is_blind(qs[r * dk]);
      if (a.causal) seen = seen && key <= p && (a.window <= 0 || key > p - a.window);
      sc[e] = seen ? s : -INFINITY;
    }
    __syncthreads();
    for (int r = warp; r < kTileRows; r += kAttThreads / 32) {
      const float s = sc[r * kKeyTile + lane];
      float top = s;
      for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float old = mx[r], now = max_nan(old, top);
      const float p = now == -INFINITY || s == -INFINITY ? 0.f : exp2f(s - now);
      float sum = p;
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sc[r * kKeyTile + lane] = p;
      __syncwarp();
      if (lane == 0) {
        const float f = old == -INFINITY ? 0.f : exp2f(old - now);
        al[r] = f, mx[r] = now, sm[r] = sm[r] * f + sum;
      }
    }
    expand_rows(a.v, a.vc, at_v, cv, kv, ld);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kMaxAcc / kTileRows; ++c) {
      const int j = tid + kAttThreads * c;
      if (j < dv) {
#pragma unroll
        for (int r = 0; r < kTileRows; ++r) acc[c * kTileRows + r] *= al[r];
        for (int t = 0; t < kKeyTile; ++t) {
          const float v = kv[t * ld + j];
          if (fabsf(v) < INFINITY) {
#pragma unroll
            for (int r = 0; r < kTileRows; ++r) acc[c * kTileRows + r] = fmaf(sc[r * kKeyTile + t], v, acc[c * kTileRows + r]);
          } else {   // a row that does not see it has weight 0, and 0 times infinity is not 0
#pragma unroll
            for (int r = 0; r < kTileRows; ++r) {
              const float p = sc[r * kKeyTile + t];
              if (p != 0.f) acc[c * kTileRows + r] = fmaf(p, v, acc[c * kTileRows + r]);
            }
          }
        }
      }
    }
  }
  __syncthreads();
  float* part = a.part + (((int64_t)blockIdx.x * a.Hkv + hk) * a.nsplit + split) * kTileRows * (dv + 2);
#pragma unroll
  for (int c = 0; c < kMaxAcc / kTileRows; ++c) {
    const int j = tid + kAttThreads * c;
    if (j < dv)
#pragma unroll
      for (int r = 0; r < kTileRows; ++r) part[r * (dv + 2) + j] = acc[c * kTileRows + r];
  }
  if (tid < kTileRows) part[tid * (dv + 2) + dv] = mx[tid], part[tid * (dv + 2) + dv + 1] = sm[tid];
}

__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == TQ_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == TQ_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Grid: (tiles, Hkv): the 8 rows of a tile: splits merged, then o = (Pi_V^T acc + c S_V^T acc_s) / sum.
__global__ void __launch_bounds__(kAppThreads) paged_combine_simt_kernel(AttnArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int R = kTileRows;
  const int d = a.v.d, m = a.v.m, dv = d + m;
  float* acc = reinterpret_cast<float*>(smem);        // [8][d], then [8][m]
  float* acc2 = acc + R * d;
  float* o1 = acc2 + R * m;                           // [8][d]
  float* o2 = o1 + R * d;
  float* part_s = o2 + R * d;
  __shared__ float f[R];
  const int tid = threadIdx.x, hk = blockIdx.y;
  const Tile tl = warp_find_tile(a.bt, a.G, R, blockIdx.x);
  if (tl.b < 0) return;
  const float* part = a.part + ((int64_t)blockIdx.x * a.Hkv + hk) * a.nsplit * R * (dv + 2);
  for (int e = tid; e < R * dv; e += kAppThreads) {
    const int r = e / dv, j = e - r * dv;
    float top = -INFINITY;
    for (int s = 0; s < a.nsplit; ++s) top = max_nan(top, part[(s * R + r) * (dv + 2) + dv]);
    float v = 0.f, sum = 0.f;
    if (top != -INFINITY)
      for (int s = 0; s < a.nsplit; ++s) {
        const float* p = part + (s * R + r) * (dv + 2);
        const float wgt = p[dv] == -INFINITY ? 0.f : exp2f(p[dv] - top);
        v = fmaf(wgt, p[j], v);
        sum = fmaf(wgt, p[dv + 1], sum);
      }
    if (j < d) acc[r * d + j] = v;
    else acc2[r * m + j - d] = v;
    if (j == 0) f[r] = sum > 0.f ? 1.f / sum : 0.f;
  }
  __syncthreads();
  rows_matvec<R>(acc, d, a.v.Pi, d, part_s, o1);      // sum_j acc_j Pi[j][i]
  if (m > 0) rows_matvec<R>(acc2, m, a.v.S, d, part_s, o2);
  const int64_t tok0 = a.bt.q_start[tl.b];
  for (int e = tid; e < R * d; e += kAppThreads) {
    const int r = e / d, i = e - r * d, row = tl.row0 + r;
    if (r >= tl.nrows) continue;
    float v = o1[e];
    if (m > 0) v = fmaf(kQjlScale / (float)m, o2[e], v);
    store_any(a.out, a.q_dtype, ((tok0 + row / a.G) * a.Hq + hk * a.G + row % a.G) * d + i, v * f[r]);
  }
}

}  // namespace paged
}  // namespace tqk
