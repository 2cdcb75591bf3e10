// Append of many vectors to paged caches on the tcgen05 tensor cores: d = 64 or 128, d signs or none.
//
// What is computed is paged_append.cuh's definition, with the same exact indices and signs. A tile is 128 rows (token, head):
//   preparation (eight warps, four lanes a row): norm, rotation, |z|, then z times a power of two that puts |z| into
//     [2^7, 2^8) as a pair of f16 (z_h + z_l holds 22 bits);
//   D1 = z Pi^T        three contractions: z_h Pi_h + z_h Pi_l + z_l Pi_h (Pi times 2^8 as an f16 pair; 16-bit vectors that
//                      need no preparation are exact in z_h and take two);
//   indices (thread = row), e = y - c[idx]; sign rows: e times 2^10 as an f16 pair into tensor memory,
//   D2 = e M^T         three contractions again, the e pair as the operand in tensor memory;
//   signs of D2.
// Bound by the preparation: its loads of positions, pages, cosines and vectors depend on one another, and one tile's places and
// vectors ahead (two without signs or at d = 64) do not hide them (tensor pipe 21 %, ALU 45 % busy). 8 heads x 16384 tokens of
// bf16 with rotation and signs, keys and values: 122 us warm, 131 cold, 9 us for each of a CTA's 14 tiles, where the bytes
// alone would take 14. The contractions are issued in a fixed order, the next tile's first before this tile's second.
// Two tiles are under way at a time, each with its own 256 columns: D1, then D2 in the same 128; e_h and e_l in the others.
//
// Exactness. A coordinate closer to a border than kTcBandY, and a sign closer to 0 than kTcBandS, is computed again by its
// warp in fp64 from the inputs. What separates D1 from the exact value, in units of u = 2^-24 and of |z| (Cauchy-Schwarz over
// the row of Pi): z in fp32 with norm and rotation at most 6, its f16 pair 2, Pi's 2, the dropped z_l Pi_l 1, the quotient
// by |z| 2 |y|; and the 24 accumulations inside the tensor cores, whose rounding is not specified. Measured against fp64
// over 6.7e7 coordinates of bf16 and fp32 vectors with outlier channels, with and without preparation: 1.0 u root mean
// square, 8.5 u at most; the band is 24 u. A sign's sum gathers d such differences with weights of length m_norm: measured
// 0.24 u m_norm root mean square and at most 2.3 u m_norm, 1.1 where the sum is below 0.2; the band is 6 u m_norm. About
// 0.4 % of the rows of 2-bit codes and 1 % of 4-bit ones have a coordinate, and 0.2 % a sign, that is computed twice.
#pragma once

#include "paged_flash.cuh"

namespace tqk {
namespace paged {

constexpr float kU = 5.9604645e-8f;
constexpr float kTcBandY = 24.f * kU;
constexpr float kTcBandS = 6.f * kU;    // times m_norm
// Warps 0-7 prepare, 8-23 finish (two groups of eight, two threads per row: the chain of one thread per row took twice as
// long), 24 issues, 25-27 fill its warpgroup. Registers: 896 threads x 72 at launch = 128 x (2 x 104 + 4 x 64 + 40).
constexpr int kTaPrepWarps = 8, kTaEpiWarps = 16;
constexpr int kTaThreads = 32 * (kTaPrepWarps + kTaEpiWarps + 4);

// f16 pairs, K-major: Pi_h, Pi_l (times 2^8), M_h, M_l (times 2^5); each D/64 slices of D rows.
template <int D, bool PROD>
struct TaLayout {
  static constexpr uint32_t kMat = (D / 64) * D * 128;
  static constexpr uint32_t kOps = (PROD ? 4 : 2) * kMat;
  static constexpr uint32_t kTile = (D / 64) * kAtomRows;         // 128 rows
  static constexpr int kStages = PROD && D == 128 ? 1 : 2;        // z tiles (pairs)
  static constexpr uint32_t kA = kOps;
  static constexpr uint32_t kRowInfo = 128 * 24;
  static constexpr uint32_t kRow = kA + kStages * 2 * kTile;      // per tile of four: int64 place[128], float2 (N_s, N)[128], int64 rp[128]
  static constexpr uint32_t kSq = kRow + 4 * kRowInfo;              // float [2 groups][2][128]: halves of |e|^2
  static constexpr uint32_t kBars = kSq + 2048;
  // op_full, a_full[2], a_empty[2], d1_full[2], e_full[2], d2_full[2], d_free[2]
  static constexpr int kNumBars = 13;
  static constexpr uint32_t kMisc = kBars + 8 * kNumBars;
  static constexpr uint32_t kBytes = kMisc + 16;
};
static_assert(TaLayout<128, true>::kBytes <= 232448 && TaLayout<128, false>::kBytes <= 232448, "shared memory of one CTA");

struct AppendTcArgs {
  const void* x;
  int64_t stride;
  int x_dtype, Hkv, exact_hi;   // exact_hi: the vectors are 16-bit and taken as they are
  Batch bt;
  Prep prep;                    // cos_sin / weight NULL for values; check_prep then holds the keys' rotation
  Prep check_prep;              // a token whose key has no rotation row is skipped on both sides
  Quant q;
  CacheView c;
  const uint8_t* ops;
  int* err;
};

// The sum of squares of a row that four lanes hold, times f^2. Eights are summed in fp32 and those in fp64: a norm stored in fp32 is off
// by half a step for the root, a quarter for this result's rounding and about 0.15 for the eights (one sum of 32 in fp32: a
// step more).
template <int C>
__device__ __forceinline__ float row_squares(const float (&z)[8 * C], float f = 1.f) {
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float p = (z[8 * c] * f) * (z[8 * c] * f);
#pragma unroll
    for (int x = 1; x < 8; ++x) p = fmaf(z[8 * c + x] * f, z[8 * c + x] * f, p);
    ss += (double)p;
  }
  ss += __shfl_xor_sync(0xffffffffu, ss, 1);
  ss += __shfl_xor_sync(0xffffffffu, ss, 2);
  return (float)ss;
}

// 1 / sqrt(mean of squares + eps) of such a row; the whole warp calls it.
template <int C>
__device__ __forceinline__ float row_rms(const float (&z)[8 * C], int d, float eps) {
  const float ss = row_squares<C>(z);
  const bool many = !(ss < kManySquares);
  if (__any_sync(0xffffffffu, many)) {
    const float s2 = row_squares<C>(z, kSmaller);
    if (many) return kSmaller / sqrtf(s2 / (float)d);
  }
  return 1.f / sqrtf(ss / (float)d + eps);
}

// Index of |y| among the positive half of a symmetric codebook (H = 2^(BITS - 1) cells, H - 1 positive borders b[1 ..]), the
// distance to the nearest border met, and the cell's centroid (positive).
template <int BITS>
struct Cells {
  static constexpr int H = 1 << (BITS - 1);
  float b[H > 1 ? H - 1 : 1], c[H];
};
template <int BITS>
__device__ __forceinline__ void find_cell(const Cells<BITS>& t, float ay, uint32_t& k, float& c, float& near) {
  if (BITS == 1) {
    k = 0, c = t.c[0];
  } else if (BITS == 2) {
    const bool o = ay > t.b[0];
    near = fminf(near, fabsf(ay - t.b[0]));
    k = o, c = o ? t.c[1] : t.c[0];
  } else if (BITS == 3) {
    const bool p = ay > t.b[1];
    const float b1 = p ? t.b[2] : t.b[0];
    const bool q = ay > b1;
    near = fminf(near, fminf(fabsf(ay - t.b[1]), fabsf(ay - b1)));
    k = 2 * p + q;
    c = p ? (q ? t.c[3] : t.c[2]) : (q ? t.c[1] : t.c[0]);
  } else {
    const bool p = ay > t.b[3];
    const float b1 = p ? t.b[5] : t.b[1];
    const bool q = ay > b1;
    const float b2 = p ? (q ? t.b[6] : t.b[4]) : (q ? t.b[2] : t.b[0]);
    const bool r = ay > b2;
    near = fminf(fminf(near, fabsf(ay - t.b[3])), fminf(fabsf(ay - b1), fabsf(ay - b2)));
    k = 4 * p + 2 * q + r;
    const float c0 = p ? (q ? t.c[6] : t.c[4]) : (q ? t.c[2] : t.c[0]);
    const float c1 = p ? (q ? t.c[7] : t.c[5]) : (q ? t.c[3] : t.c[1]);
    c = r ? c1 : c0;
  }
}

// The warp's lanes compute Pi_j z (and |z|) of the row (token t, head h) in fp64; every lane gets both.
template <int D>
__device__ __forceinline__ void exact_row(const AppendTcArgs& a, int64_t t, int h, int64_t rp, double (&z)[D / 32], double& n) {
  prep_head<double, D / 32>(a.x, a.x_dtype, t * a.stride + (int64_t)h * D, D, a.prep, rp, z);
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) ss += z[c] * z[c];
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  n = sqrt(ss);
}
template <int D>
__device__ __forceinline__ void load_row64(const double* row, double (&p)[D / 32]) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) p[c] = __ldg(row + (threadIdx.x & 31) + 32 * c);
}
template <int D>
__device__ __forceinline__ double exact_dot(const double (&p)[D / 32], const double (&z)[D / 32]) {
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s += p[c] * z[c];
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// 16 columns of this thread's tensor-memory lane, waited for; 8 columns stored.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int D, int BITS, bool PROD>
__global__ void __launch_bounds__(kTaThreads, 1) paged_append_tc_kernel(AppendTcArgs a) {
  using L = TaLayout<D, PROD>;
  extern __shared__ __align__(1024) unsigned char smem_tiles[];
  unsigned char* const smem = smem_tiles;
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t rows = a.bt.ntok * a.Hkv;
  const int ntiles = (int)((rows + 127) / 128);
  const int mine = ntiles > (int)blockIdx.x ? (ntiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  const uint32_t bars = base + L::kBars, op_full = bars;
  auto a_full = [&](int s) { return bars + 8u * (1 + s); };
  auto a_empty = [&](int s) { return bars + 8u * (3 + s); };
  auto d1_full = [&](int g) { return bars + 8u * (5 + g); };
  auto e_full = [&](int g) { return bars + 8u * (7 + g); };
  auto d2_full = [&](int g) { return bars + 8u * (9 + g); };
  auto d_free = [&](int g) { return bars + 8u * (11 + g); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  grid_dep_launch();
  if ((base & 1023u) != 0) {
    if (tid == 0) report_error(a.err, kErrInternal);
    return;
  }
  if (tid == 0) {
    *abort_flag = 0;
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + L::kBars);
    for (int i = 0; i < L::kNumBars; ++i) {
      const int n = i == 1 || i == 2 ? kTaPrepWarps : i == 7 || i == 8 || i == 11 || i == 12 ? kTaEpiWarps / 2 : 1;
      bar_init(b + i, n);
    }
  }
  constexpr int kMmaWarp = kTaPrepWarps + kTaEpiWarps;
  if (warp == kMmaWarp) {
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

  if (warp < kTaPrepWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
    // ---- rows -> z pairs; lane q of a row's four holds the 16-byte chunks (8 coordinates) q, q + 4, ...
    constexpr int C = D / 32;
    const int ql = lane & 3, rot = a.prep.cos_sin ? a.prep.rot_dim : 0, half = rot >> 1;
    const int64_t start0 = a.bt.q_start[0], end = a.bt.q_start[a.bt.B];
    for (int i = 0; i < mine; ++i) {
      const int s = i % L::kStages, ri = i & 3;
      int64_t* place_s = reinterpret_cast<int64_t*>(smem + L::kRow + ri * L::kRowInfo);
      float2* norm_s = reinterpret_cast<float2*>(smem + L::kRow + ri * L::kRowInfo + 1024);
      int64_t* rp_s = reinterpret_cast<int64_t*>(smem + L::kRow + ri * L::kRowInfo + 2048);   // for the rows that are computed twice
      // places and (16-bit) values of both halves first: one latency for them all
      int64_t at2[2], rp2[2], from2[2];
      uint4 raw[2][C];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t row = ((int64_t)blockIdx.x + (int64_t)i * gridDim.x) * 128 + k * 64 + warp * 8 + (lane >> 2);
        int64_t t;
        int h;
        split_row(row, a.Hkv, t, h);
        int64_t at = -1, rp = 0;
        from2[k] = t * a.stride + (int64_t)h * D;
        const bool in = row < rows && t >= start0 && t < end;
        if (a.x_dtype != TQ_F32) {
#pragma unroll
          for (int c = 0; c < C; ++c)
            raw[k][c] = in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + from2[k] + 8 * (ql + 4 * c)))
                           : make_uint4(0, 0, 0, 0);
        }
        if (in) {
          const int b = last_at_or_before(a.bt.q_start, a.bt.B, (int)t);
          const int64_t p = (int64_t)a.bt.len[b] - a.bt.q_start[b + 1] + t;
          at = place_of(a.bt, b, p, h, a.Hkv);
          if (a.check_prep.cos_sin) {
            rp = a.check_prep.pos ? (int64_t)a.check_prep.pos[t] : p;
            if (rp < 0 || rp >= a.check_prep.max_pos) at = -1;
          }
          if (at < 0 && ql == 0) report_error(a.err, kErrPaged);
        }
        at2[k] = at, rp2[k] = rp;
      }
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const int r = k * 64 + warp * 8 + (lane >> 2);
        const int64_t at = k ? at2[1] : at2[0], rp = k ? rp2[1] : rp2[0], from = k ? from2[1] : from2[0];
        const bool ok = at >= 0;
        float z[8 * C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (a.x_dtype == TQ_F32) {
            const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + from + 8 * (ql + 4 * c));
            const float4 v = ok ? __ldg(src) : make_float4(0, 0, 0, 0), w = ok ? __ldg(src + 1) : make_float4(0, 0, 0, 0);
            z[8 * c] = v.x, z[8 * c + 1] = v.y, z[8 * c + 2] = v.z, z[8 * c + 3] = v.w;
            z[8 * c + 4] = w.x, z[8 * c + 5] = w.y, z[8 * c + 6] = w.z, z[8 * c + 7] = w.w;
          } else {
            const uint4 w = k ? raw[1][c] : raw[0][c];
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = a.x_dtype == TQ_F16 ? etc::pair_to_float2<true>(x[e]) : etc::pair_to_float2<false>(x[e]);
              z[8 * c + 2 * e] = v.x, z[8 * c + 2 * e + 1] = v.y;
            }
          }
        }
        float rms = 1.f;
        if (a.prep.weight) {
          rms = row_rms<C>(z, D, a.prep.eps);
#pragma unroll
          for (int x = 0; x < 8 * C; ++x)
            z[x] *= rms * load_any(a.prep.weight, a.prep.weight_dtype, 8 * (ql + 4 * (x >> 3)) + (x & 7));
        }
        if (ok && rot) {
          const float* cs = a.prep.cos_sin + rp * rot;
          if (rot == D && !a.prep.interleaved) {
#pragma unroll
            for (int c = 0; c < C / 2; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k0 = 8 * (ql + 4 * c) + 4 * e;
                const float4 co = *reinterpret_cast<const float4*>(cs + k0);
                const float4 si = *reinterpret_cast<const float4*>(cs + D / 2 + k0);
                const float cc[4] = {co.x, co.y, co.z, co.w}, sn[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  float& lo = z[8 * c + 4 * e + x];
                  float& hi = z[8 * (c + C / 2) + 4 * e + x];
                  const float p = lo, w = hi;
                  lo = p * cc[x] - w * sn[x], hi = w * cc[x] + p * sn[x];
                }
              }
          } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int k0 = 8 * (ql + 4 * c) + 2 * e;
                float& y0 = z[8 * c + 2 * e];
                float& y1 = z[8 * c + 2 * e + 1];
                if (k0 < rot && a.prep.interleaved) {
                  const float co = cs[k0 >> 1], si = cs[half + (k0 >> 1)], p = y0, w = y1;
                  y0 = p * co - w * si, y1 = w * co + p * si;
                } else if (k0 < rot) {   // the partner may be any lane's: read again
                  const int kk = k0 < half ? k0 : k0 - half, other = k0 < half ? k0 + half : k0 - half;
                  const float sg = k0 < half ? -1.f : 1.f;
                  float p0 = load_any(a.x, a.x_dtype, from + other), p1 = load_any(a.x, a.x_dtype, from + other + 1);
                  if (a.prep.weight) {
                    p0 *= rms * load_any(a.prep.weight, a.prep.weight_dtype, other);
                    p1 *= rms * load_any(a.prep.weight, a.prep.weight_dtype, other + 1);
                  }
                  y0 = y0 * cs[kk] + sg * p0 * cs[half + kk];
                  y1 = y1 * cs[kk + 1] + sg * p1 * cs[half + kk + 1];
                }
              }
          }
        }
        float ss = row_squares<C>(z);
        float n = sqrtf(ss);
        const bool odd = !(ss >= 1e-30f && ss < 1e37f);
        if (__any_sync(0xffffffffu, odd)) {   // squares out of fp32's range: once more about the largest coordinate
          float top = 0.f;
#pragma unroll
          for (int x = 0; x < 8 * C; ++x) top = fmaxf(top, fabsf(z[x]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          int e = 0;
          if (top > 0.f && top < INFINITY) frexpf(top, &e);
          const float dn1 = ldexpf(1.f, -e / 2), dn2 = ldexpf(1.f, -e - -e / 2);
          ss = 0.f;
#pragma unroll
          for (int x = 0; x < 8 * C; ++x) {
            const float w = z[x] * dn1 * dn2;
            ss = fmaf(w, w, ss);
          }
          ss += __shfl_xor_sync(0xffffffffu, ss, 1);
          ss += __shfl_xor_sync(0xffffffffu, ss, 2);
          if (odd) n = ldexpf(sqrtf(ss), e);
        }
        int e = 0;
        if (n > 0.f && n < INFINITY) frexpf(n, &e);
        if (k == 0 && i >= L::kStages) wait(a_empty(s), (i / L::kStages - 1) & 1);
        const float sc1 = ldexpf(1.f, (8 - e) / 2), sc2 = ldexpf(1.f, (8 - e) - (8 - e) / 2);   // 2^(8 - e) in two steps: no overflow
        const uint32_t zr = base + L::kA + s * 2 * L::kTile + r * 128;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float v0 = z[8 * c + 2 * x] * sc1 * sc2, v1 = z[8 * c + 2 * x + 1] * sc1 * sc2;
            hi[x] = half2_bits(v0, v1);
            const float2 back = etc::pair_to_float2<true>(hi[x]);
            lo[x] = half2_bits(v0 - back.x, v1 - back.y);
          }
          const int ch = ql + 4 * c;
          const uint32_t off = (ch >> 3) * kAtomRows + (((ch & 7) ^ (r & 7)) << 4);
          sts128(zr + off, hi[0], hi[1], hi[2], hi[3]);
          if (!a.exact_hi) sts128(zr + L::kTile + off, lo[0], lo[1], lo[2], lo[3]);
        }
        if (ql == 0) place_s[r] = at, rp_s[r] = rp, norm_s[r] = make_float2(n * sc1 * sc2, n);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(a_full(s));
    }
  } else if (warp > kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
    const uint32_t lead = elect_one();
    if (lead) {
      expect_tx(op_full, L::kOps);
      for (uint32_t o = 0; o < L::kOps; o += L::kMat) bulk_load(base + o, a.ops + o, L::kMat, op_full);
    }
    wait(op_full, 0);
    const uint64_t a_desc = sw128_desc(base + L::kA), b_desc = sw128_desc(base);
    constexpr uint32_t kT16 = L::kTile >> 4, kM16 = L::kMat >> 4, kI = flash_idesc(D, false);
    auto first = [&](int i) {
      const int s = i % L::kStages, g = i & 1;
      wait(a_full(s), (i / L::kStages) & 1);
      if (i >= 2) wait(d_free(g), (i / 2 - 1) & 1);
      tc_fence_after();
      const uint64_t zh = a_desc + s * 2 * kT16, zl = zh + kT16;
      const uint32_t d = tmem + 256 * g;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t ao = ((c >> 2) * kAtomRows + (c & 3) * 32) >> 4, bo = ((c >> 2) * (D * 128) + (c & 3) * 32) >> 4;
        if (c == 0) mma_ss<false>(lead, d, zh + ao, b_desc + bo, kI);
        else mma_ss<true>(lead, d, zh + ao, b_desc + bo, kI);
        mma_ss<true>(lead, d, zh + ao, b_desc + kM16 + bo, kI);
        if (!a.exact_hi) mma_ss<true>(lead, d, zl + ao, b_desc + bo, kI);
      }
      commit_one(lead, d1_full(g));
      commit_one(lead, a_empty(s));
    };
    if (mine > 0) first(0);
    for (int i = 0; i < mine; ++i) {
      if (i + 1 < mine) first(i + 1);
      if (PROD) {
        const int g = i & 1;
        wait(e_full(g), (i / 2) & 1);
        tc_fence_after();
        const uint32_t d = tmem + 256 * g, eh = d + 128, el = eh + D / 2;
        const uint64_t mh = b_desc + 2 * kM16, ml = b_desc + 3 * kM16;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t bo = ((c >> 2) * (D * 128) + (c & 3) * 32) >> 4;
          mma_ts(lead, d, eh + 8 * c, mh + bo, kI, c > 0 ? 1u : 0u);
          mma_ts(lead, d, eh + 8 * c, ml + bo, kI, 1u);
          mma_ts(lead, d, el + 8 * c, mh + bo, kI, 1u);
        }
        commit_one(lead, d2_full(g));
      }
    }
    // tensor memory is released below: the last contractions must have ended
    for (int i = max(0, mine - 2); i < mine; ++i) {
      (void)wait_bar(d1_full(i & 1), (i / 2) & 1);
      if (PROD) (void)wait_bar(d2_full(i & 1), (i / 2) & 1);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    // ---- indices and signs: thread = half a row of the group's tiles
    const int ew = warp - kTaPrepWarps, g = ew >> 3, part = (ew >> 2) & 1, r = (ew & 3) * 32 + lane;
    float* const sq = reinterpret_cast<float*>(smem + L::kSq) + 256 * g + r;
    const uint32_t col = tmem + 256 * g + ((uint32_t)((ew & 3) * 32) << 16);
    Cells<BITS> cells;
#pragma unroll
    for (int i = 0; i < Cells<BITS>::H; ++i) cells.c[i] = a.q.cent[Cells<BITS>::H + i];
#pragma unroll
    for (int i = 0; i < Cells<BITS>::H - 1; ++i) cells.b[i] = a.q.bnd[Cells<BITS>::H + i];
    for (int i = g; i < mine; i += 2) {
      const int ri = i & 3;
      wait(d1_full(g), (i / 2) & 1);
      tc_fence_after();
      const int64_t at = reinterpret_cast<const int64_t*>(smem + L::kRow + ri * L::kRowInfo)[r];
      const float2 nn = reinterpret_cast<const float2*>(smem + L::kRow + ri * L::kRowInfo + 1024)[r];
      const int64_t row0 = ((int64_t)blockIdx.x + (int64_t)i * gridDim.x) * 128;
      const float inv = nn.x > 0.f ? 0.00390625f / nn.x : 0.f;   // 2^-8 / |z scaled|
      const bool some = at >= 0 && nn.x > 0.f && nn.x < INFINITY;
      // a row in fp64: its token, head and rotation position again
      auto fetch_exact = [&](int who, double (&z)[D / 32], double& n) {
        int64_t t;
        int h;
        split_row(row0 + (ew & 3) * 32 + who, a.Hkv, t, h);
        const int64_t rp = reinterpret_cast<const int64_t*>(smem + L::kRow + ri * L::kRowInfo + 2048)[(ew & 3) * 32 + who];
        exact_row<D>(a, t, h, rp, z, n);
      };
      float esq[2] = {0.f, 0.f};
      uint64_t front = 0;
#pragma unroll 1   // 16 coordinates at a time: the unrolled row would not stay in the instruction cache
      for (int c16 = part * (D / 32); c16 < (part + 1) * (D / 32); ++c16) {
        uint32_t v[16];
        tmem_ld16(col + 16 * c16, v);
        float near, err[PROD ? 16 : 1];
        uint64_t w;
        auto cells_of = [&](bool mask_only) -> uint32_t {
          uint32_t close = 0;
          near = INFINITY, w = 0;
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float y = __uint_as_float(v[x]);
            uint32_t k;
            float c, d = fabsf(y);
            find_cell<BITS>(cells, fabsf(y), k, c, d);
            if (mask_only) {
              close |= some && d <= kTcBandY ? 1u << x : 0u;
              continue;
            }
            near = fminf(near, d);
            const bool pos = y > 0.f;
            const uint32_t idx = pos ? Cells<BITS>::H + k : Cells<BITS>::H - 1 - k;
            w |= (uint64_t)idx << (x * BITS);
            if (PROD) {
              const float e = nn.x > 0.f ? y - (pos ? c : -c) : 0.f;
              err[x & (PROD ? 15 : 0)] = e;
            }
          }
          return close;
        };
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * inv);
        cells_of(false);
        if (__any_sync(0xffffffffu, some && near <= kTcBandY)) {
          // which coordinates: a mask per lane, then one after the other by the whole warp
          const uint32_t close = cells_of(true);
          for (unsigned todo = __ballot_sync(0xffffffffu, close != 0); todo; todo &= todo - 1) {
            const int who = __ffs(todo) - 1;
            double z[D / 32], n, p[D / 32];
            uint32_t m = __shfl_sync(0xffffffffu, close, who);
            load_row64<D>(a.q.Pi64() + (size_t)(16 * c16 + __ffs(m) - 1) * D, p);   // under way while the row is prepared
            fetch_exact(who, z, n);
            for (; m; m &= m - 1) {
              const int x = __ffs(m) - 1;
              const double y = exact_dot<D>(p, z) / n;
              if (m & (m - 1)) load_row64<D>(a.q.Pi64() + (size_t)(16 * c16 + __ffs(m & (m - 1)) - 1) * D, p);
              int k = 0;
              for (int q = 0; q < (1 << BITS) - 1; ++q) k += a.q.bnd64()[q] < y;
              // the fp32 value nearest to y for which the comparisons above give k: a positive cell holds its upper border
              // there, a negative one its lower
              const float lo = k > 0 ? a.q.bnd[k - 1] : -2.f, hi = k < (1 << BITS) - 1 ? a.q.bnd[k] : 2.f;
              float yf = (float)y;
              if (k >= Cells<BITS>::H) {
                if (yf <= lo) yf = lo > 0.f ? __int_as_float(__float_as_int(lo) + 1) : 1e-30f;
                yf = fminf(yf, hi);
              } else {
                if (yf >= hi) yf = hi < 0.f ? __int_as_float(__float_as_int(hi) + 1) : 0.f;
                yf = fmaxf(yf, lo);
              }
#pragma unroll
              for (int q = 0; q < 16; ++q) v[q] = q == x && lane == who ? __float_as_uint(yf) : v[q];
            }
          }
          cells_of(false);
        }
        if ((c16 & 1) == 0) {
          front = w;
        } else if (at >= 0) {   // 32 coordinates: BITS words
          uint8_t* dst = a.c.codes + at * a.q.codes_B + 2 * BITS * (c16 - 1);
          if (BITS == 4) {
            *reinterpret_cast<uint4*>(dst) = make_uint4((uint32_t)front, (uint32_t)(front >> 32), (uint32_t)w, (uint32_t)(w >> 32));
          } else if (BITS == 2) {
            *reinterpret_cast<uint2*>(dst) = make_uint2((uint32_t)front, (uint32_t)w);
          } else if (BITS == 1) {
            *reinterpret_cast<uint32_t*>(dst) = (uint32_t)front | (uint32_t)w << 16;
          } else {
            uint32_t* d32 = reinterpret_cast<uint32_t*>(dst);
            d32[0] = (uint32_t)front;
            d32[1] = (uint32_t)(front >> 32) | (uint32_t)w << 16;
            d32[2] = (uint32_t)(w >> 16);
          }
        }
        if (PROD) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float r0 = err[PROD ? 2 * x : 0], r1 = err[PROD ? 2 * x + 1 : 0];
            esq[0] = fmaf(r0, r0, esq[0]), esq[1] = fmaf(r1, r1, esq[1]);
            const float e0 = r0 * 1024.f, e1 = r1 * 1024.f;
            hi[x] = half2_bits(e0, e1);
            const float2 back = etc::pair_to_float2<true>(hi[x]);
            lo[x] = half2_bits(e0 - back.x, e1 - back.y);
          }
          tmem_st8(col + 128 + 8 * c16, hi);
          tmem_st8(col + 128 + D / 2 + 8 * c16, lo);
        }
      }
      if (at >= 0 && part == 0) store_norm(a.c.norms, a.q.norm_dtype, at, (double)nn.y);
      if (!PROD) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(d_free(g));
        continue;
      }
      sq[128 * part] = esq[0] + esq[1];
      etc::tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(e_full(g));
      wait(d2_full(g), (i / 2) & 1);   // both halves of the group have arrived before: sums and codes are there
      tc_fence_after();
      if (at >= 0 && part == 0) a.c.rnorms[at] = __double2half((double)nn.y * sqrt((double)sq[0] + (double)sq[128]));
      const float band = kTcBandS * a.q.m_norm * 32768.f;   // D2 comes times 2^5 2^10
      uint32_t first_half = 0;
#pragma unroll 1
      for (int c16 = part * (D / 32); c16 < (part + 1) * (D / 32); ++c16) {
        uint32_t v[16];
        tmem_ld16(col + 16 * c16, v);
        uint32_t sg = 0;
        float near = INFINITY;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float d = __uint_as_float(v[x]);
          sg |= d >= 0.f ? 1u << x : 0u;
          near = fminf(near, fabsf(d));
        }
        if (__any_sync(0xffffffffu, some && near <= band)) {
          uint32_t close = 0;
#pragma unroll
          for (int x = 0; x < 16; ++x)
            if (some && fabsf(__uint_as_float(v[x])) <= band) close |= 1u << x;
          for (unsigned todo = __ballot_sync(0xffffffffu, close != 0); todo; todo &= todo - 1) {
            const int who = __ffs(todo) - 1;
            double z[D / 32], n, cz[D / 32];
            fetch_exact(who, z, n);
            // the row's indices, from its codes (stored by this warp, above)
            const uint32_t* cw = reinterpret_cast<const uint32_t*>(a.c.codes + __shfl_sync(0xffffffffu, at, who) * a.q.codes_B);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) cz[c] = a.q.cent64()[packed_field(cw, lane + 32 * c, BITS)];
            for (uint32_t m = __shfl_sync(0xffffffffu, close, who); m; m &= m - 1) {
              const int x = __ffs(m) - 1, j = 16 * c16 + x;
              double p[D / 32], q[D / 32];
              load_row64<D>(a.q.S64() + (size_t)j * D, p);
              load_row64<D>(a.q.M64() + (size_t)j * D, q);
              const double d = exact_dot<D>(p, z) / n - exact_dot<D>(q, cz);
              if (lane == who) sg = d >= 0.0 ? sg | 1u << x : sg & ~(1u << x);
            }
          }
        }
        if ((c16 & 1) == 0) first_half = sg;
        else if (at >= 0)
          reinterpret_cast<uint32_t*>(a.c.signs + at * a.q.signs_B)[c16 >> 1] = nn.x > 0.f ? first_half | sg << 16 : 0xffffffffu;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(d_free(g));
    }
  }
  grid_dep_wait();   // the keys' kernel, if this one was started beside it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u) : "memory");
}

}  // namespace paged
}  // namespace tqk
