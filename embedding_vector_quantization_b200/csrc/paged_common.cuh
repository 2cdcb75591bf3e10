// What the paged kernels share: the ragged batch, places in the pages, and the preparation of a head (RMS norm,
// then the rotation by its position) in fp64 and fp32.
#pragma once

#include "common.cuh"

namespace tqk {
namespace paged {

// tq_paged_batch, tq_head_prep and tq_paged_cache as the kernels take them.
struct Batch {
  const int32_t* q_start;
  const int32_t* len;
  const int32_t* table;
  int B, max_pages, page_size, max_q;
  int64_t ntok, num_pages;
};

struct Prep {
  const float* cos_sin;
  const int32_t* pos;
  const void* weight;
  int64_t max_pos;
  int rot_dim, interleaved, weight_dtype;
  float eps;
};

struct CacheView {
  uint8_t* codes;
  uint8_t* signs;
  void* norms;
  __half* rnorms;
};

// A handle's constants.
struct Quant {
  int d, bits, m, norm_dtype, codes_B, signs_B;
  const float *PiT, *Pi, *MT, *ST, *S, *cent, *bnd;
  const double* t64;
  float m_abs, m_norm, cent_up;
  __device__ const double* Pi64() const { return t64; }
  __device__ const double* S64() const { return t64 + (size_t)d * d; }
  __device__ const double* M64() const { return t64 + (size_t)d * d + (size_t)m * d; }
  __device__ const double* bnd64() const { return t64 + (size_t)d * d + (size_t)2 * m * d; }
  __device__ const double* cent64() const { return bnd64() + 16; }
};

// The sequence of token row t (-1: padding, or before the first): every lane of the warp counts a share of the
// sequences that end at or before t.
__device__ __forceinline__ int warp_find_seq(const Batch& bt, int64_t t) {
  const int lane = threadIdx.x & 31;
  int ended = 0;
  for (int i = lane; i < bt.B; i += 32) ended += (int64_t)bt.q_start[i + 1] <= t;
  ended = __reduce_add_sync(0xffffffffu, ended);
  if (ended >= bt.B || t < bt.q_start[0]) return -1;
  return ended;
}

// Token rows of sequence b; none if its bounds lie outside the batch's rows or hold more than max_q, which grids and workspaces
// are made for.
__device__ __forceinline__ int seq_tokens(const Batch& bt, int b) {
  const int lo = bt.q_start[b], hi = bt.q_start[b + 1];
  return lo >= 0 && hi > lo && hi <= bt.ntok && hi - lo <= bt.max_q ? hi - lo : 0;
}

// Whether attention leaves sequence b out for such bounds, or some of its keys because the table is too narrow for its length.
__device__ __forceinline__ bool seq_cut_short(const Batch& bt, int b) {
  const int lo = bt.q_start[b], hi = bt.q_start[b + 1];
  return hi != lo && (seq_tokens(bt, b) == 0 || bt.len[b] > (int64_t)bt.max_pages * bt.page_size);
}

// Token and head of row `row` = token * H + head (a 64-bit quotient only where 32 bits do not do).
__device__ __forceinline__ void split_row(int64_t row, int H, int64_t& t, int& h) {
  if (row <= 0xffffffffll) {
    const uint32_t q = (uint32_t)row / (uint32_t)H;
    t = q, h = (int)((uint32_t)row - q * H);
  } else {
    t = row / H, h = (int)(row - t * H);
  }
}

// Row index of (position p, head h) of sequence b in a cache [page][Hkv][slot], -1 if its page is out of range.
__device__ __forceinline__ int64_t place_of(const Batch& bt, int b, int64_t p, int h, int Hkv) {
  if (p < 0 || p >= (int64_t)bt.max_pages * bt.page_size) return -1;
  const uint32_t pi = (uint32_t)p / (uint32_t)bt.page_size, slot = (uint32_t)p - pi * bt.page_size;   // p < 2^30
  const int64_t page = bt.table[(int64_t)b * bt.max_pages + pi];
  if (page < 0 || page >= bt.num_pages) return -1;
  return (page * Hkv + h) * bt.page_size + slot;
}

// The larger one, NaN if either is: a row's running maximum takes a NaN score along, and everything after it becomes NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Squares above this are summed again of vectors times 2^-70 (exact): the sum of 256 stays within fp32. eps is nothing to them.
constexpr float kManySquares = 1e37f;
constexpr float kSmaller = 8.4703295e-22f;   // 2^-70

// The warp's lanes prepare one head x[0 .. d) (d <= 256): lane l holds coordinates l, l + 32, ... in z[]. T is
// double where a code's exact index is at stake, float for queries. p: the rotation position (checked by the caller).
template <typename T, int MAXC>
__device__ __forceinline__ void prep_head(const void* x, int x_dtype, int64_t at, int d, const Prep& pr, int64_t p,
                                          T (&z)[MAXC]) {
  const int lane = threadIdx.x & 31;
  T ss = 0;
#pragma unroll
  for (int c = 0; c < MAXC; ++c) {
    const int i = lane + 32 * c;
    z[c] = i < d ? (T)load_any(x, x_dtype, at + i) : (T)0;
    ss += z[c] * z[c];
  }
  if (pr.weight) {
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    T r = (T)1 / sqrt(ss / (T)d + (T)pr.eps);
    if (sizeof(T) == 4 && !(ss < (T)kManySquares)) {   // the whole warp's
      ss = 0;
#pragma unroll
      for (int c = 0; c < MAXC; ++c) ss += (z[c] * (T)kSmaller) * (z[c] * (T)kSmaller);
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      r = (T)kSmaller / sqrt(ss / (T)d);
    }
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
      const int i = lane + 32 * c;
      if (i < d) z[c] = z[c] * r * (T)load_any(pr.weight, pr.weight_dtype, i);
    }
  }
  if (!pr.cos_sin) return;
  const int half = pr.rot_dim >> 1;
  const float* cs = pr.cos_sin + p * pr.rot_dim;
  if (pr.interleaved) {   // the partner of coordinate i is i ^ 1: the neighbouring lane
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
      const T other = __shfl_xor_sync(0xffffffffu, z[c], 1);
      const int i = lane + 32 * c;
      if (i < pr.rot_dim) {
        const T co = (T)cs[i >> 1], si = (T)cs[half + (i >> 1)];
        z[c] = (i & 1) ? z[c] * co + other * si : z[c] * co - other * si;
      }
    }
    return;
  }
  // the partner is half a rotation away: any lane and any chunk, fetched from a copy of all of z
  T y[MAXC];
#pragma unroll
  for (int c = 0; c < MAXC; ++c) {
    const int i = lane + 32 * c;
    const int j = i < half ? i + half : i - half;
    T other = 0;
#pragma unroll
    for (int e = 0; e < MAXC; ++e) {
      const T v = __shfl_sync(0xffffffffu, z[e], j & 31);
      if ((j >> 5) == e) other = v;
    }
    y[c] = z[c];
    if (i < pr.rot_dim) {
      const int k = i < half ? i : i - half;
      const T co = (T)cs[k], si = (T)cs[half + k];
      y[c] = i < half ? z[c] * co - other * si : z[c] * co + other * si;
    }
  }
#pragma unroll
  for (int c = 0; c < MAXC; ++c) z[c] = y[c];
}

// A prepared head whose products with S (128 of a few each) could pass fp32 is taken times 2^-64; returns what makes up for it. The
// whole warp calls it.
template <int MAXC>
__device__ __forceinline__ float tame_head(float (&z)[MAXC]) {
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < MAXC; ++c) top = fmaxf(top, fabsf(z[c]));
  if (!__any_sync(0xffffffffu, top > 1e30f)) return 1.f;
#pragma unroll
  for (int c = 0; c < MAXC; ++c) z[c] *= 5.421011e-20f;
  return 1.8446744e19f;
}

}  // namespace paged
}  // namespace tqk
