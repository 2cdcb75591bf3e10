// Append of a ragged batch's keys and values to paged caches, any format: the general kernel.
//
// Per vector: z = the head after its norm and rotation, N = |z|, y = Pi z / N, idx_j = #{i : beta_i < y_j}; prod rows:
// e = y - c[idx], sigma_j = [(M e)_j >= 0] with M = S Pi^T, rnorm = N |e| ("Google TurboQuant: 6x KV-cache compression",
// "Stage 1" and "Stage 2").
//
// The indices and signs are exact. y is computed in fp32 with a proven error bound and every coordinate closer than
// that to a border is computed again in fp64 from fp64 tables, a warp per coordinate:
//   y: products summed in chunks of 32 fused multiply-adds, then over the chunks. With u = 2^-24 each chunk sum is off by
//      at most 32 u sum |Pi z|, the sum over C <= 8 chunks by C u more, and z and Pi carry u each from their own rounding:
//      |dy| <= (32 + C + 2 + 1) u sum |Pi_ji z_i| / N <= 43 u (Cauchy-Schwarz: rows of Pi and z / N have length 1). The
//      quotient by N and the fp32 border cost 2 u |y| <= 2 u more: kBandY = 46 u = 2.8e-6.
//   sigma: |d(M e)_j| <= sum_i |M_ji| |de_i| + 43 u sum |M_ji e_i| <= m_abs (kBandY + 2 u) + 43 u m_norm |e|, with m_abs
//      and m_norm the largest row of M in the 1-norm and the 2-norm, and |e| <= 1. The exact value is then taken as
//      (S z)_j / N - (M c[idx])_j: two dot products, no further rotation.
// At d = 128 about 5e-4 of the 4-bit indices and 6e-4 of the signs are computed twice.
//
// Bound by latency where rows are few (32 tokens of 4 heads, keys and values: 18 us, 25 with signs) and by fp32 products
// from shared memory where they are many (16384 tokens of 8 heads with signs: 1.8 ms, 0.13 on the tensor cores).
#pragma once

#include "paged_common.cuh"

namespace tqk {
namespace paged {

constexpr float kBandY = 46.f * 5.9604645e-8f;
constexpr int kAppThreads = 256;

struct AppendArgs {
  const void* x[2];       // keys, values
  int64_t stride[2];
  int x_dtype, Hkv;
  Batch bt;
  Prep prep;              // keys only
  Quant q[2];
  CacheView c[2];
  int* err;
};

__host__ __device__ inline size_t append_smem_bytes(int d, int m, int R, int threads) {
  const int w = d > m ? d : m;
  return (size_t)R * d * 8 + 2 * (size_t)R * w * 4 + (size_t)R * w + (size_t)threads * R * 4 + 64;
}

// out[r][j] = sum_i in[r][i] T[i][j] for the CTA's R rows: thread (j, part) sums its share of i in chunks of 32.
template <int R, int NT = kAppThreads>
__device__ __forceinline__ void rows_matvec(const float* in, int ni, const float* T, int nj, float* part_s, float* out) {
  constexpr int kStep = NT > 256 ? 16 : 32;   // chunk; the bound above holds for chunks of 32 and less
  const int tid = threadIdx.x;
  const int parts = max(1, min(NT / nj, ni / kStep));
  const int j = tid % nj, part = tid / nj;
  float acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = 0.f;
  if (part < parts) {
    const int chunks = ni / kStep;
    for (int c = part; c < chunks; c += parts) {
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
      const float* t = T + (size_t)(kStep * c) * nj + j;
#pragma unroll 16
      for (int i = 0; i < kStep; ++i) {
        const float p = __ldg(t + (size_t)i * nj);
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = fmaf(in[r * ni + kStep * c + i], p, s[r]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] += s[r];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) part_s[(r * parts + part) * nj + j] = acc[r];
  }
  __syncthreads();
  for (int e = tid; e < R * nj; e += NT) {
    const int r = e / nj, jj = e - r * nj;
    float s = 0.f;
    for (int p = 0; p < parts; ++p) s += part_s[(r * parts + p) * nj + jj];
    out[e] = s;
  }
  __syncthreads();
}

// Grid: (row groups of R, 2): y = 0 keys, 1 values; row = token * Hkv + head. d <= 32 MAXC. One row and 1024 threads where latency counts
// (the products' loads are then all under way at once), eight rows and 256 threads where there are many.
template <int R, int NT, int MAXC>
__global__ void __launch_bounds__(NT) paged_append_kernel(AppendArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int kind = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Quant& Q = a.q[kind];
  const int d = Q.d, m = Q.m, w = max(d, m), bits = Q.bits;
  double* zd = reinterpret_cast<double*>(smem);                  // [R][d]
  float* zf = reinterpret_cast<float*>(zd + (size_t)R * d);      // [R][w] z, then e
  float* ys = zf + (size_t)R * w;                                // [R][w] y, then M e
  float* part_s = ys + (size_t)R * w;                            // [256 R]
  uint8_t* idx = reinterpret_cast<uint8_t*>(part_s + (size_t)NT * R);   // [R][w] indices, then signs
  __shared__ int64_t place[R];
  __shared__ double nrm[R], cd[16], bd[16];
  __shared__ float cf[16], bf[16];
  __shared__ float esum[R];

  if (tid < 16) {
    bd[tid] = Q.bnd64()[tid], cd[tid] = Q.cent64()[tid];
    bf[tid] = (float)bd[tid], cf[tid] = (float)cd[tid];
  }
  const int64_t row0 = (int64_t)blockIdx.x * R, rows = a.bt.ntok * a.Hkv;
  for (int r = warp; r < R; r += NT / 32) {
    const int64_t row = row0 + r;
    int64_t t;
    int h;
    split_row(row, a.Hkv, t, h);
    const int b = row < rows ? warp_find_seq(a.bt, t) : -1;
    int64_t at = -1, rp = 0;
    bool bad = false;
    if (b >= 0) {
      const int64_t p = (int64_t)a.bt.len[b] - a.bt.q_start[b + 1] + t;
      at = place_of(a.bt, b, p, h, a.Hkv);
      if (kind == 0 && a.prep.cos_sin) {
        rp = a.prep.pos ? (int64_t)a.prep.pos[t] : p;
        if (rp < 0 || rp >= a.prep.max_pos) at = -1;
      }
      // a value's key may have been refused for its rotation: both rows of the token are skipped together
      if (kind == 1 && a.prep.cos_sin) {
        const int64_t rk = a.prep.pos ? (int64_t)a.prep.pos[t] : p;
        if (rk < 0 || rk >= a.prep.max_pos) at = -1;
      }
      bad = at < 0;
    }
    if (bad && lane == 0) report_error(a.err, kErrPaged);
    double z[MAXC];
#pragma unroll
    for (int c = 0; c < MAXC; ++c) z[c] = 0.0;
    double ss = 0.0;
    if (at >= 0) {
      Prep pr = a.prep;
      if (kind == 1) pr.cos_sin = nullptr, pr.weight = nullptr;
      prep_head<double, MAXC>(a.x[kind], a.x_dtype, t * a.stride[kind] + (int64_t)h * d, d, pr, rp, z);
    }
#pragma unroll
    for (int c = 0; c < MAXC; ++c)
      if (lane + 32 * c < d) {
        zd[r * d + lane + 32 * c] = z[c];
        zf[r * d + lane + 32 * c] = (float)z[c];
        ss += z[c] * z[c];
      }
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) place[r] = at, nrm[r] = sqrt(ss), esum[r] = 0.f;
  }
  __syncthreads();
  bool any = false;
#pragma unroll
  for (int r = 0; r < R; ++r) any |= place[r] >= 0;
  if (!any) return;

  rows_matvec<R, NT>(zf, d, Q.PiT, d, part_s, ys);
  // indices; a coordinate within the band of a border is computed again by the whole warp
  for (int e0 = warp * 32; e0 < R * d; e0 += NT) {   // d % 32 = 0: the warp stays in one row
    const int e = e0 + lane, r = e / d;
    const double n = nrm[r];
    float y = n > 0.0 ? ys[e] / (float)n : 0.f;
    int k = 0;
    bool close = false;
    for (int i = 0; i < (1 << bits) - 1; ++i) {
      k += bf[i] < y;
      close |= fabsf(bf[i] - y) <= kBandY;
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, close && n > 0.0); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1, j = e0 + who - r * d;
      double s = 0.0;
      for (int i = lane; i < d; i += 32) s += Q.Pi64()[(size_t)j * d + i] * zd[r * d + i];
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == who) {
        s /= n;
        k = 0;
        for (int i = 0; i < (1 << bits) - 1; ++i) k += bd[i] < s;
        y = (float)s;
      }
    }
    idx[e] = (uint8_t)k;
    const float err = n > 0.0 ? y - cf[k] : 0.f;
    zf[e] = err;                 // e: every read of z (fp32) is behind the product's barrier
    if (m > 0) {
      float q = err * err;
      for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      if (lane == 0) ys[e0] = q;   // this warp's own columns of y, read above
    }
  }
  __syncthreads();
  if (m > 0 && tid < R) {
    float s = 0.f;
    for (int c = 0; c < d; c += 32) s += ys[tid * d + c];   // a fixed order
    esum[tid] = s;
  }
  // codes: word by word, LSB first
  const int cw = Q.codes_B / 4;
  for (int e = tid; e < R * cw; e += NT) {
    const int r = e / cw, wd = e - r * cw;
    if (place[r] < 0) continue;
    uint32_t v = 0;
    for (int j = (32 * wd) / bits; j < d && j * bits < 32 * wd + 32; ++j) {
      const int sh = j * bits - 32 * wd;
      v |= sh >= 0 ? (uint32_t)idx[r * d + j] << sh : (uint32_t)idx[r * d + j] >> -sh;
    }
    reinterpret_cast<uint32_t*>(a.c[kind].codes + place[r] * Q.codes_B)[wd] = v;
  }
  if (tid < R && place[tid] >= 0) store_norm(a.c[kind].norms, Q.norm_dtype, place[tid], nrm[tid]);
  if (m == 0) return;
  __syncthreads();
  if (tid < R && place[tid] >= 0 && bits > 0)
    a.c[kind].rnorms[place[tid]] = __double2half(nrm[tid] * sqrt((double)esum[tid]));
  rows_matvec<R, NT>(zf, d, Q.MT, m, part_s, ys);
  const float band = Q.m_abs * (kBandY + 1.2e-7f) + 43.f * 5.9604645e-8f * Q.m_norm;
  for (int e0 = warp * 32; e0 < R * m; e0 += NT) {
    const int e = e0 + lane, r = e / m;
    const double n = nrm[r];
    bool pos = ys[e] >= 0.f;
    for (unsigned todo = __ballot_sync(0xffffffffu, fabsf(ys[e]) <= band && n > 0.0); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1, j = e0 + who - r * m;
      double s = 0.0, q = 0.0;
      for (int i = lane; i < d; i += 32) {
        s += Q.S64()[(size_t)j * d + i] * zd[r * d + i];
        q += Q.M64()[(size_t)j * d + i] * cd[idx[r * d + i]];
      }
      s = s / n - q;
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == who) pos = s >= 0.0;
    }
    const unsigned word = __ballot_sync(0xffffffffu, n > 0.0 ? pos : true);
    if (lane == 0 && place[r] >= 0)
      reinterpret_cast<uint32_t*>(a.c[kind].signs + place[r] * Q.signs_B)[(e0 - r * m) >> 5] = word;
  }
}

}  // namespace paged
}  // namespace tqk
