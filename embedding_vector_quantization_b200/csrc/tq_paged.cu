// C ABI of the paged operators (declared in include/tq.h): argument checks, workspace layout and launches of
// tq_append_paged and tq_attn_paged.

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "tq.h"
#include "internal.h"
#include "common.cuh"
#include "paged_common.cuh"
#include "paged_append.cuh"
#include "paged_attn_simt.cuh"
#include "paged_flash.cuh"
#include "paged_decode.cuh"
#include "paged_append_tc.cuh"

namespace {

using namespace tqk::paged;

#define fail tq_internal_fail

struct Nvtx {
  explicit Nvtx(const char* n) { nvtxRangePushA(n); }
  ~Nvtx() { nvtxRangePop(); }
};

// The handle's device for the duration of a call.
struct DeviceGuard {
  int was = -1;
  cudaError_t err = cudaSuccess;
  explicit DeviceGuard(int dev) {
    int cur = 0;
    err = cudaGetDevice(&cur);
    if (err == cudaSuccess && cur != dev) {
      err = cudaSetDevice(dev);
      if (err == cudaSuccess) was = cur;
    }
  }
  ~DeviceGuard() {
    if (was >= 0) cudaSetDevice(was);
  }
};

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int elem_bytes(int dt) { return dt == TQ_F32 ? 4 : 2; }
bool valid_dtype(int dt) { return dt == TQ_F32 || dt == TQ_F16 || dt == TQ_BF16; }

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TQ_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  return tq_internal_ok();
}

// Raises a kernel's shared memory limit once per device.
template <typename K>
int allow_smem(K kernel, size_t bytes, int device, std::atomic<uint64_t>& seen) {
  if (device >= 0 && device < 64 && (seen.load(std::memory_order_acquire) >> device & 1)) return TQ_OK;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return fail(TQ_ECUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  if (device >= 0 && device < 64) seen.fetch_or(1ull << device, std::memory_order_release);
  return TQ_OK;
}

Quant quant_of(const tq_view& v) {
  Quant q{};
  q.d = v.d, q.bits = v.bits, q.m = v.m, q.norm_dtype = v.norm_dtype, q.codes_B = v.codes_B, q.signs_B = v.signs_B;
  q.PiT = v.PiT, q.Pi = v.Pi, q.MT = v.MT, q.ST = v.ST, q.S = v.S, q.cent = v.cent, q.bnd = v.bnd, q.t64 = v.t64;
  q.m_abs = v.m_abs, q.m_norm = v.m_norm, q.cent_up = v.cent_up;
  return q;
}

int check_handles(const tq_handle* hk, const tq_handle* hv, tq_view* k, tq_view* v) {
  if (!hk || !hv) return fail(TQ_EINVAL, "handle is NULL");
  tq_internal_view(hk, k);
  tq_internal_view(hv, v);
  if (k->polar || v->polar) return fail(TQ_EUNSUPPORTED, "polar handles have no paged operators");
  if (k->d != v->d) return fail(TQ_EINVAL, "key d=%d, value d=%d", k->d, v->d);
  if (k->d > 256 || k->m > 256 || v->m > 256) return fail(TQ_EUNSUPPORTED, "paged operators need d <= 256 and m <= 256");
  if (k->device != v->device) return fail(TQ_EINVAL, "the handles are on devices %d and %d", k->device, v->device);
  return TQ_OK;
}

// What can be said of a cache without its handle.
int check_pages(const tq_paged_cache* c, const char* name) {
  if (!c) return fail(TQ_EINVAL, "%s cache is NULL", name);
  if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16)
    return fail(TQ_EINVAL, "%s page_size=%d (a multiple of 16, 16..1024)", name, c->page_size);
  if (c->num_pages < 1 || c->num_pages > (int64_t)1 << 31) return fail(TQ_EINVAL, "%s num_pages=%lld", name, (long long)c->num_pages);
  if (!c->norms) return fail(TQ_EINVAL, "%s cache: NULL norms", name);
  if (!aligned(c->norms, 16) || !aligned(c->codes, 16) || !aligned(c->signs, 16) || !aligned(c->rnorms, 16))
    return fail(TQ_EINVAL, "%s cache: pointers need 16-byte alignment", name);
  return TQ_OK;
}

int check_pages(const tq_paged_cache* k, const tq_paged_cache* v) {
  int st;
  if ((st = check_pages(k, "key")) || (st = check_pages(v, "value"))) return st;
  if (k->page_size != v->page_size || k->num_pages != v->num_pages)
    return fail(TQ_EINVAL, "the key and value caches share one block table: page_size and num_pages must agree");
  return TQ_OK;
}

int check_cache(const tq_view& h, const tq_paged_cache* c, const char* name) {
  if (h.codes_B > 0 && !c->codes) return fail(TQ_EINVAL, "%s cache: NULL codes", name);
  if (h.m > 0 && (!c->signs || (h.bits > 0 && !c->rnorms))) return fail(TQ_EINVAL, "%s cache: prod rows need signs and rnorms", name);
  return TQ_OK;
}

int check_batch(const tq_paged_batch* b, const tq_paged_cache* k, Batch* out) {
  if (!b) return fail(TQ_EINVAL, "batch is NULL");
  if (b->B < 0 || b->B > 65536) return fail(TQ_EINVAL, "B=%d outside 0..65536", b->B);
  if (b->ntok < 0 || b->ntok > (1 << 24)) return fail(TQ_EINVAL, "ntok=%lld outside 0..2^24", (long long)b->ntok);
  if (b->max_pages < 1 || (int64_t)b->max_pages * (k ? k->page_size : 1) > 0x40000000)
    return fail(TQ_EINVAL, "max_pages=%d (at least 1, at most 2^30 positions)", b->max_pages);
  if (b->max_q < 0 || b->max_q > b->ntok) return fail(TQ_EINVAL, "max_q=%d outside 0..ntok", b->max_q);
  if (b->B > 0 && (!b->q_start || !b->len || !b->block_table)) return fail(TQ_EINVAL, "batch: NULL array");
  if (!aligned(b->q_start, 4) || !aligned(b->len, 4) || !aligned(b->block_table, 4)) return fail(TQ_EINVAL, "batch: misaligned array");
  out->q_start = b->q_start, out->len = b->len, out->table = b->block_table;
  out->B = b->B, out->max_pages = b->max_pages, out->max_q = b->max_q, out->ntok = b->ntok;
  out->page_size = k ? k->page_size : 16, out->num_pages = k ? k->num_pages : 0;
  return TQ_OK;
}

int check_prep(const tq_head_prep* p, Prep* out) {
  *out = Prep{};
  if (!p) return TQ_OK;
  if (p->cos_sin) {
    if (p->rot_dim < 8 || p->rot_dim % 8) return fail(TQ_EINVAL, "rot_dim=%d (a multiple of 8, 8..d)", p->rot_dim);
    if (p->max_pos < 1) return fail(TQ_EINVAL, "max_pos=%lld", (long long)p->max_pos);
    if (p->interleaved != 0 && p->interleaved != 1) return fail(TQ_EINVAL, "interleaved=%d (0 or 1)", p->interleaved);
    if (!aligned(p->cos_sin, 16) || !aligned(p->pos, 4)) return fail(TQ_EINVAL, "cos_sin or pos misaligned");
    out->cos_sin = p->cos_sin, out->pos = p->pos, out->max_pos = p->max_pos, out->rot_dim = p->rot_dim;
    out->interleaved = p->interleaved;
  }
  if (p->weight) {
    if (!valid_dtype(p->weight_dtype)) return fail(TQ_EINVAL, "weight dtype %d", p->weight_dtype);
    if (!(p->eps > 0.f) || !std::isfinite(p->eps)) return fail(TQ_EINVAL, "eps must be positive");
    if (!aligned(p->weight, elem_bytes(p->weight_dtype))) return fail(TQ_EINVAL, "weight misaligned");
    out->weight = p->weight, out->weight_dtype = p->weight_dtype, out->eps = p->eps;
  }
  return TQ_OK;
}

int check_rows(const void* x, int dtype, int64_t stride, int H, int d, const char* name) {
  if (!x) return fail(TQ_EINVAL, "%s is NULL", name);
  if (!aligned(x, 16)) return fail(TQ_EINVAL, "%s misaligned (16 bytes)", name);
  if (stride < (int64_t)H * d || stride * elem_bytes(dtype) % 16) return fail(TQ_EINVAL, "%s stride %lld", name, (long long)stride);
  return TQ_OK;
}

CacheView view_of(const tq_view& h, const tq_paged_cache* c) {
  CacheView v{};
  v.codes = h.codes_B > 0 ? c->codes : nullptr;
  v.signs = h.m > 0 ? c->signs : nullptr;
  v.norms = c->norms;
  v.rnorms = h.m > 0 && h.bits > 0 ? static_cast<__half*>(c->rnorms) : nullptr;
  return v;
}

int device_sms(int device) {
  static std::atomic<int> sms[64];
  if (device < 0 || device >= 64) return 148;
  int n = sms[device].load();
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) n = 148;
    sms[device].store(n);
  }
  return n;
}

// ---------------------------------------------------------------- append

template <int R, int NT, int MAXC>
int append_simt(const AppendArgs& a, int device, cudaStream_t s) {
  static std::atomic<uint64_t> seen{0};
  if (int st = allow_smem(paged_append_kernel<R, NT, MAXC>, append_smem_bytes(256, 256, R, NT), device, seen)) return st;
  const int m = std::max(a.q[0].m, a.q[1].m);
  const unsigned groups = (unsigned)((a.bt.ntok * a.Hkv + R - 1) / R);
  tq_launch_scope scope("append_paged", s);
  paged_append_kernel<R, NT, MAXC><<<dim3(groups, 2), NT, append_smem_bytes(a.q[0].d, m, R, NT), s>>>(a);
  return launched("paged_append_kernel");
}

bool simt_forced() {
  const char* e = std::getenv("TQ_SIMT");
  return e && std::strcmp(e, "1") == 0;
}

// A launch that may start while the kernel before it drains (that kernel's results are read after griddepcontrol.wait).
template <typename K, typename A>
int launch_after(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const A& args, const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
  if (e != cudaSuccess) return fail(TQ_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  return launched(what);
}

template <int D, int BITS, bool PROD>
int append_tc_launch(const AppendTcArgs& a, int device, bool beside, cudaStream_t s) {
  static std::atomic<uint64_t> seen{0};
  using L = TaLayout<D, PROD>;
  if (int st = allow_smem(paged_append_tc_kernel<D, BITS, PROD>, L::kBytes, device, seen)) return st;
  const int64_t tiles = (a.bt.ntok * a.Hkv + 127) / 128;
  const dim3 grid((unsigned)std::min<int64_t>(tiles, std::max(1, device_sms(device) / 2)));   // keys and values run side by side
  tq_launch_scope scope("append_paged", s);
  if (beside) return launch_after(paged_append_tc_kernel<D, BITS, PROD>, grid, kTaThreads, L::kBytes, s, a, "paged_append_tc_kernel");
  paged_append_tc_kernel<D, BITS, PROD><<<grid, kTaThreads, L::kBytes, s>>>(a);
  return launched("paged_append_tc_kernel");
}

template <int D, bool PROD>
int append_tc_bits(const AppendTcArgs& a, int device, bool beside, cudaStream_t s) {
  switch (a.q.bits) {
    case 1: return append_tc_launch<D, 1, PROD>(a, device, beside, s);
    case 2: return append_tc_launch<D, 2, PROD>(a, device, beside, s);
    case 3: return append_tc_launch<D, 3, PROD>(a, device, beside, s);
    default: return append_tc_launch<D, 4, PROD>(a, device, beside, s);
  }
}

// Keys on one half of the SMs, values on the other: the second kernel starts beside the first and waits for it before it ends.
int append_tc(const AppendArgs& g, const tq_view& k, const tq_view& v, cudaStream_t s) {
  for (int kind = 0; kind < 2; ++kind) {
    const tq_view& w = kind ? v : k;
    AppendTcArgs a{};
    a.x = g.x[kind], a.stride = g.stride[kind], a.x_dtype = g.x_dtype, a.Hkv = g.Hkv, a.bt = g.bt;
    a.check_prep = g.prep;
    if (kind == 0) a.prep = g.prep;
    a.exact_hi = g.x_dtype != TQ_F32 && !a.prep.cos_sin && !a.prep.weight;
    a.q = g.q[kind], a.c = g.c[kind], a.ops = w.ops_app, a.err = g.err;
    int st;
    if (w.d == 128) st = w.m ? append_tc_bits<128, true>(a, w.device, kind == 1, s) : append_tc_bits<128, false>(a, w.device, kind == 1, s);
    else st = w.m ? append_tc_bits<64, true>(a, w.device, kind == 1, s) : append_tc_bits<64, false>(a, w.device, kind == 1, s);
    if (st) return st;
  }
  return TQ_OK;
}

// ---------------------------------------------------------------- attention, general kernels

struct SimtPlan {
  int64_t tiles;      // upper bound over the batches that fit the arguments
  int nsplit;
  size_t qr, part, total;
};

SimtPlan simt_plan(const tq_view& k, const tq_view& v, const Batch& b, int Hq, int Hkv, int sms) {
  SimtPlan p{};
  const int G = Hq / Hkv;
  p.tiles = std::min<int64_t>(b.ntok * G / kTileRows + b.B, (int64_t)b.B * (((int64_t)b.max_q * G + kTileRows - 1) / kTileRows));
  p.tiles = std::max<int64_t>(p.tiles, 1);
  const int64_t keys = (int64_t)b.max_pages * b.page_size;
  p.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>((8 * sms) / (p.tiles * Hkv), (keys + 255) / 256));
  p.qr = 0;
  p.part = up((size_t)b.ntok * Hq * (k.d + k.m) * 4, 256);
  // tiles * Hkv * nsplit <= max(tiles * Hkv, 8 sms): a smaller batch never needs more than a larger one
  p.total = p.part + up((size_t)std::max<int64_t>(p.tiles * Hkv, 8 * sms) * kTileRows * (v.d + v.m + 2) * 4, 256) + 256;
  return p;
}

int attn_simt(AttnArgs& a, const tq_view& k, const tq_view& v, const SimtPlan& p, char* ws, int device, cudaStream_t s) {
  static std::atomic<uint64_t> s1{0}, s2{0}, s3{0};
  constexpr int R = 8;
  const size_t combine = (size_t)R * (256 + 256 + 2 * 256) * 4 + (size_t)kAppThreads * R * 4;
  int st;
  if ((st = allow_smem(paged_qprep_kernel<R>, qprep_smem_bytes(256, 256, R), device, s1)) ||
      (st = allow_smem(paged_attn_simt_kernel, attn_simt_smem_bytes(512, 512), device, s2)) ||
      (st = allow_smem(paged_combine_simt_kernel, combine, device, s3)))
    return st;
  a.qr = reinterpret_cast<float*>(ws + p.qr);
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.nsplit = p.nsplit;
  {
    tq_launch_scope scope("paged_qprep", s);
    paged_qprep_kernel<R><<<(unsigned)((a.bt.ntok * a.Hq + R - 1) / R), kAppThreads, qprep_smem_bytes(k.d, k.m, R), s>>>(a);
  }
  if ((st = launched("paged_qprep_kernel"))) return st;
  {
    tq_launch_scope scope("paged_attn", s);
    paged_attn_simt_kernel<<<dim3((unsigned)p.tiles, (unsigned)a.Hkv, (unsigned)p.nsplit), kAttThreads,
                             attn_simt_smem_bytes(k.d + k.m, v.d + v.m), s>>>(a);
  }
  if ((st = launched("paged_attn_simt_kernel"))) return st;
  tq_launch_scope scope("paged_combine", s);
  paged_combine_simt_kernel<<<dim3((unsigned)p.tiles, (unsigned)a.Hkv), kAppThreads, combine, s>>>(a);
  return launched("paged_combine_simt_kernel");
}

// ---------------------------------------------------------------- attention of chunks, tensor cores

// 16-bit queries, d = 64 or 128, d signs or none (those handles hold the operands).
bool flash_formats(const tq_view& k, const tq_view& v) { return k.ops16k && v.ops16v && !simt_forced(); }

struct FlashPlan {
  int64_t max_seqs, max_tiles, max_items;
  int heads, ctas;      // KV heads of a round
  size_t head, tile_start, item_start, unit, ke, ve, kn, vn, seen, part, krows, vrows, qrows, qfactor, total;
};

constexpr size_t kRowsCap = (size_t)1 << 30;   // f16 rows held at a time, unless one KV head needs more

// other: whether sequences with up to 8 query rows of a KV head go elsewhere (those with more may, which changes no size).
FlashPlan flash_plan(const tq_view& k, const Batch& b, int Hq, int Hkv, bool other, int sms) {
  FlashPlan p{};
  const int64_t G = Hq / Hkv;
  p.max_seqs = std::min<int64_t>(b.B, std::min(b.ntok, other ? b.ntok * G / 9 : b.ntok));
  p.max_tiles = std::max<int64_t>(1, p.max_seqs * (((int64_t)b.max_pages * b.page_size + kKT - 1) / kKT));
  p.max_items = std::max<int64_t>(1, b.ntok * G / kItemRows + p.max_seqs);
  const size_t tile = (size_t)(k.d / 64) * kAtomRows;
  p.heads = (int)std::max<size_t>(1, std::min<size_t>(Hkv, kRowsCap / (2 * tile * (size_t)p.max_tiles)));
  // Sizes that grow with every argument, unlike heads: a smaller batch never needs more.
  const size_t rows = std::min((size_t)Hkv * p.max_tiles * tile, std::max(kRowsCap / 2, (size_t)p.max_tiles * tile));
  p.ctas = sms;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = up(at + bytes, 256);
    return here;
  };
  p.head = take(16);
  p.tile_start = take((size_t)(b.B + 1) * 4);
  p.item_start = take((size_t)(b.B + 1) * 4);
  p.unit = take((size_t)(p.max_items + 1) * 4);
  p.ke = take((size_t)Hkv * p.max_tiles * 4);
  p.ve = take((size_t)Hkv * p.max_tiles * 4);
  p.kn = take(rows / tile * kKT * 4);
  p.vn = take(rows / tile * kKT * 4);
  p.seen = take((size_t)p.max_tiles * 16);
  p.part = take((size_t)2 * p.ctas * kItemRows * (k.d + 4) * 4);
  p.krows = take(rows);
  p.vrows = take(rows);
  p.qrows = take((size_t)Hkv * p.max_items * 2 * tile);
  p.qfactor = take((size_t)Hkv * p.max_items * kItemRows * 4);
  p.total = at + 256;
  return p;
}

template <int D>
int attn_flash(const AttnArgs& g, const tq_view& k, const tq_view& v, const FlashPlan& p, int small_rows, bool behind, char* ws,
               cudaStream_t s) {
  static std::atomic<uint64_t> s1{0}, s2{0};
  int st;
  if ((st = allow_smem(paged_expand_kernel<D>, ExLayout<D>::kBytes, k.device, s1)) ||
      (st = allow_smem(paged_flash_kernel<D>, FlLayout<D>::kBytes, k.device, s2)))
    return st;
  FlashArgs a{};
  a.q = g.q, a.q_stride = g.q_stride, a.q_dtype = g.q_dtype, a.Hq = g.Hq, a.Hkv = g.Hkv, a.G = g.G;
  a.bt = g.bt, a.prep = g.prep, a.kq = g.k, a.vq = g.v, a.kc = g.kc, a.vc = g.vc, a.kops = k.ops16k, a.vops = v.ops16v;
  a.scale = g.scale, a.causal = g.causal, a.window = g.window, a.small_rows = small_rows, a.ctas = p.ctas;
  a.out = g.out, a.err = g.err;
  auto ints = [&](size_t off) { return reinterpret_cast<int*>(ws + off); };
  a.p.head = ints(p.head), a.p.tile_start = ints(p.tile_start), a.p.item_start = ints(p.item_start), a.p.unit = ints(p.unit);
  a.p.ke = ints(p.ke), a.p.ve = ints(p.ve);
  a.p.kn = reinterpret_cast<float*>(ws + p.kn), a.p.vn = reinterpret_cast<float*>(ws + p.vn), a.p.seen = reinterpret_cast<uint32_t*>(ws + p.seen);
  a.p.part = reinterpret_cast<float*>(ws + p.part);
  a.p.krows = reinterpret_cast<uint8_t*>(ws + p.krows), a.p.vrows = reinterpret_cast<uint8_t*>(ws + p.vrows);
  a.p.qrows = reinterpret_cast<uint8_t*>(ws + p.qrows), a.p.qfactor = reinterpret_cast<float*>(ws + p.qfactor);
  a.p.max_tiles = (int)p.max_tiles, a.p.max_items = (int)p.max_items;
  for (a.head0 = 0; a.head0 < a.Hkv; a.head0 += p.heads) {
    a.heads = std::min(p.heads, a.Hkv - a.head0);
    if (a.head0 == 0) {   // one plan serves every round
      tq_launch_scope scope("paged_plan", s);
      // Only behind another kernel of this call: a call's first kernel starts when all work before it is done.
      if (behind) {
        if ((st = launch_after(paged_plan_kernel, dim3(1), kPlanThreads, 0, s, a, "paged_plan_kernel"))) return st;
      } else {
        paged_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
        if ((st = launched("paged_plan_kernel"))) return st;
      }
    }
    {
      tq_launch_scope scope("paged_expand", s);
      if ((st = launch_after(paged_expand_kernel<D>, dim3(2 * ((p.ctas + 1) / 2)), kExThreads, ExLayout<D>::kBytes, s, a, "paged_expand_kernel"))) return st;
    }
    {
      tq_launch_scope scope("paged_qtile", s);
      if ((st = launch_after(paged_qtile_kernel<D>, dim3(8 * (unsigned)p.max_items, a.heads), kQtThreads, 0, s, a, "paged_qtile_kernel"))) return st;
    }
    {
      tq_launch_scope scope("paged_flash", s);
      if ((st = launch_after(paged_flash_kernel<D>, dim3(p.ctas), kFlThreads, FlLayout<D>::kBytes, s, a, "paged_flash_kernel"))) return st;
    }
    tq_launch_scope scope("paged_merge", s);
    if ((st = launch_after(paged_flash_merge_kernel<D>, dim3(p.ctas, D / 16), kItemRows, 0, s, a, "paged_flash_merge_kernel"))) return st;
  }
  return st;
}

// ---------------------------------------------------------------- attention of single tokens

// Query rows of a sequence and KV head up to which the single-token kernel takes them, eight at a time (each eight reads the
// packed rows again; the chunks' kernels expand them once, whatever the rows). Measured at 4 KV heads, d = 128, for 1 to 64
// sequences of 512 to 32768 tokens, against the chunks' kernels: 4-bit codes 8 rows 31..130 us to 58..817, 32 rows 37..427
// (174 to 158 in one case of six), 48 rows up to 246 to 158; with signs 16 rows 46..473 to 60..891, 24 rows up to 223 to 174.
int small_rows(const tq_view& k) { return k.m > 0 ? 16 : 32; }

// Whether the single-token kernel has these formats: 4- or 2-bit codes, signs on both sides or on neither.
bool decode_formats(const tq_view& k, const tq_view& v, const Batch& b, int Hkv) {
  if (!flash_formats(k, v) || k.norm_dtype != v.norm_dtype || b.B > kDcMaxB) return false;
  if (b.num_pages * Hkv * (b.page_size / kChunk) > 0xffffffffll) return false;   // its chunk numbers have 32 bits
  if (k.m > 0 || v.m > 0) return k.m == k.d && v.m == v.d && k.bits == 2 && v.bits == 2;
  return (k.bits == 4 && (v.bits == 4 || v.bits == 2)) || (k.bits == 2 && v.bits == 2);
}

struct DecodePlan {
  int ctas, rows;   // rows: the most that a sequence and KV head have here, a multiple of 8
  int64_t strips;    // eights of rows, at most
  bool one;
  size_t qr, part, total;
};

DecodePlan decode_plan(const tq_view& k, const tq_view& v, const Batch& b, int Hq, int Hkv, int sms) {
  DecodePlan p{};
  p.ctas = 2 * sms;
  p.rows = (int)std::min<int64_t>(small_rows(k), up((size_t)b.max_q * (Hq / Hkv), 8));
  const int64_t heads = (int64_t)b.B * Hkv;
  p.strips = heads * (p.rows / 8);
  p.qr = 0;
  p.part = up((size_t)p.strips * 8 * (k.d + k.m) * 4, 256);
  p.total = p.part + up(((size_t)p.ctas + (size_t)p.strips) * 8 * (v.d + v.m + 2) * 4, 256) + 256;
  // The tables' width may tell that every sequence is short enough for one CTA: then one kernel does it all, for as many
  // rows as the CTAs hold (16 sequences x 12 heads of 512 keys, d = 64: 24 us, 51 with more, 47 on the chunks' kernels).
  p.one = (int64_t)b.max_pages * b.page_size <= kWholeChunks * kChunk && heads <= p.ctas;
  if (p.one) {
    p.rows = (int)std::min<int64_t>(p.rows, p.ctas / heads * 8);
    p.strips = heads * (p.rows / 8);
  }
  return p;
}

template <int D, int BK, int BV, bool SG, bool NF16, bool ONE>
int decode_launch_as(const DecodeArgs& a, int device, cudaStream_t s) {
  static std::atomic<uint64_t> seen{0};
  using L = DcLayout<D, BK, BV, SG>;
  constexpr auto kernel = paged_decode_kernel<D, BK, BV, SG, NF16, ONE>;
  if (int st = allow_smem(kernel, L::bytes(kDcMaxB), device, seen)) return st;
  tq_launch_scope scope("paged_decode", s);
  if (!ONE) return launch_after(kernel, dim3(a.ctas), kDcThreads, L::bytes(a.a.bt.B), s, a, "paged_decode_kernel");
  kernel<<<a.ctas, kDcThreads, L::bytes(a.a.bt.B), s>>>(a);   // the call's first kernel
  return launched("paged_decode_kernel");
}

template <int D, int BK, int BV, bool SG, bool NF16>
int decode_launch(const DecodeArgs& a, bool one, int device, cudaStream_t s) {
  return one ? decode_launch_as<D, BK, BV, SG, NF16, true>(a, device, s) : decode_launch_as<D, BK, BV, SG, NF16, false>(a, device, s);
}

template <int D, bool NF16>
int decode_formats_launch(const DecodeArgs& a, bool one, int device, cudaStream_t s) {
  if (a.a.k.m > 0) return decode_launch<D, 2, 2, true, NF16>(a, one, device, s);
  if (a.a.k.bits == 2) return decode_launch<D, 2, 2, false, NF16>(a, one, device, s);
  return a.a.v.bits == 4 ? decode_launch<D, 4, 4, false, NF16>(a, one, device, s) : decode_launch<D, 4, 2, false, NF16>(a, one, device, s);
}

int attn_decode_paged(AttnArgs a, const tq_view& k, const tq_view& v, const DecodePlan& p, char* ws, cudaStream_t s) {
  static std::atomic<uint64_t> s1{0};
  const size_t merge = (size_t)(8 * 256 + 8 * 256 + 512 + 9 * p.ctas) * 4;
  int st;
  if ((st = allow_smem(paged_decode_merge_kernel, merge, k.device, s1))) return st;
  a.qr = reinterpret_cast<float*>(ws + p.qr);
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.small_rows = p.rows;
  DecodeArgs da{};
  da.a = a, da.ctas = p.ctas;
  const bool one = p.one;
  if (one) {
    da.ctas = (int)p.strips;
  } else {
    tq_launch_scope scope("paged_qprep", s);
    paged_qslice_kernel<<<dim3((unsigned)p.strips, (k.d + k.m) / 32), 256, 0, s>>>(da);
    if ((st = launched("paged_qslice_kernel"))) return st;
  }
  const bool h = k.norm_dtype == TQ_F16;
  if (k.d == 128) st = h ? decode_formats_launch<128, true>(da, one, k.device, s) : decode_formats_launch<128, false>(da, one, k.device, s);
  else st = h ? decode_formats_launch<64, true>(da, one, k.device, s) : decode_formats_launch<64, false>(da, one, k.device, s);
  if (st || one) return st;
  tq_launch_scope scope("paged_dmerge", s);
  return launch_after(paged_decode_merge_kernel, dim3((unsigned)a.bt.B, (unsigned)(a.Hkv * (p.rows / 8)), k.d / 32), 256, merge, s, da,
                      "paged_decode_merge_kernel");
}

// What the paths of a call may need. The single tokens' space lies before the chunks': their kernels may overlap.
size_t attn_workspace(const tq_view& k, const tq_view& v, const Batch& b, int Hq, int Hkv) {
  const int sms = device_sms(k.device);
  size_t n = 0;
  if (flash_formats(k, v)) {
    const bool other = decode_formats(k, v, b, Hkv);
    Batch fewer = b;   // no smaller batch needs more
    fewer.B = std::min(b.B, kDcMaxB);
    if (decode_formats(k, v, fewer, Hkv)) n += decode_plan(k, v, fewer, Hq, Hkv, sms).total;
    if (!other || (int64_t)b.max_q * (Hq / Hkv) > 8) n += flash_plan(k, b, Hq, Hkv, other, sms).total;
  }
  return std::max(n, simt_plan(k, v, b, Hq, Hkv, sms).total);
}

}  // namespace

extern "C" {

int tq_append_paged(const tq_handle* hk, const tq_handle* hv, const void* k_new, const void* v_new, int x_dtype,
                    int64_t k_stride, int64_t v_stride, int Hkv, const tq_paged_batch* batch, const tq_head_prep* prep,
                    const tq_paged_cache* k, const tq_paged_cache* v, void* stream) {
  Nvtx nvtx("tq_append_paged");
  tq_view kw, vw;
  AppendArgs a{};
  int st;
  if (Hkv < 1 || Hkv > 1024) return fail(TQ_EINVAL, "Hkv=%d outside 1..1024", Hkv);
  if (!valid_dtype(x_dtype)) return fail(TQ_EINVAL, "x dtype %d", x_dtype);
  if ((st = check_pages(k, v)) || (st = check_batch(batch, k, &a.bt)) || (st = check_prep(prep, &a.prep))) return st;
  if ((st = check_handles(hk, hv, &kw, &vw)) || (st = check_cache(kw, k, "key")) || (st = check_cache(vw, v, "value"))) return st;
  if (a.prep.rot_dim > kw.d) return fail(TQ_EINVAL, "rot_dim=%d, d=%d", a.prep.rot_dim, kw.d);
  if (batch->B == 0 || batch->ntok == 0) return tq_internal_ok();
  if ((st = check_rows(k_new, x_dtype, k_stride, Hkv, kw.d, "k_new")) || (st = check_rows(v_new, x_dtype, v_stride, Hkv, kw.d, "v_new")))
    return st;
  if (tq_internal_fault("launch")) return fail(TQ_ECUDA, "injected launch failure (TQ_FAULT=launch)");
  DeviceGuard dev(kw.device);
  if (dev.err != cudaSuccess) return fail(TQ_ECUDA, "device %d: %s", kw.device, cudaGetErrorString(dev.err));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = tq_internal_pre_launch(hk, s))) return st;
  a.x[0] = k_new, a.x[1] = v_new, a.stride[0] = k_stride, a.stride[1] = v_stride;
  a.x_dtype = x_dtype, a.Hkv = Hkv;
  a.q[0] = quant_of(kw), a.q[1] = quant_of(vw);
  a.c[0] = view_of(kw, k), a.c[1] = view_of(vw, v);
  a.err = kw.err;
  const int64_t rows = batch->ntok * Hkv;
  // While all rows of keys and values run at once, each with 1024 threads, that is quickest: at d = 128, 144 rows of 4-bit codes
  // take 18.5 us, 19.4 on the tensor cores and 22.6 with eight rows to a CTA; 160 rows 24.6, 20.5 and 22.6 (at d = 64 the
  // sides meet at 64 rows: 12 us both; 96 rows 16 and 14). More go to the tensor cores, where they have the format (4096
  // rows: 21 us, 45 otherwise), else eight to a CTA.
  const bool few = rows <= device_sms(kw.device) / (kw.d <= 64 ? 2 : 1);
  if (!few && kw.ops_app && vw.ops_app && !simt_forced()) return append_tc(a, kw, vw, s);
  if (kw.d <= 128) return few ? append_simt<1, 1024, 4>(a, kw.device, s) : append_simt<8, kAppThreads, 4>(a, kw.device, s);
  return few ? append_simt<1, 1024, 8>(a, kw.device, s) : append_simt<8, kAppThreads, 8>(a, kw.device, s);
}

size_t tq_attn_paged_workspace_bytes(const tq_handle* hk, const tq_handle* hv, const tq_paged_batch* batch, int Hq, int Hkv,
                                     const tq_paged_cache* k) {
  tq_view kw, vw;
  Batch b{};
  if (check_handles(hk, hv, &kw, &vw) || check_pages(k, "key") || Hkv < 1 || Hq < 1 || Hq % Hkv || check_batch(batch, k, &b)) return 0;
  return attn_workspace(kw, vw, b, Hq, Hkv);
}

int tq_attn_paged(const tq_handle* hk, const tq_handle* hv, const void* q, int q_dtype, int64_t q_stride, int Hq, int Hkv,
                  const tq_paged_batch* batch, const tq_head_prep* prep, const tq_paged_cache* k, const tq_paged_cache* v,
                  float scale, int causal, int window, void* out, void* workspace, size_t ws_bytes, void* stream) {
  Nvtx nvtx("tq_attn_paged");
  tq_view kw, vw;
  AttnArgs a{};
  int st;
  if (Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq % Hkv || Hq / Hkv > 256) return fail(TQ_EINVAL, "Hq=%d Hkv=%d", Hq, Hkv);
  if (!valid_dtype(q_dtype)) return fail(TQ_EINVAL, "q dtype %d", q_dtype);
  if (!std::isfinite(scale)) return fail(TQ_EINVAL, "scale is not finite");
  if (causal != 0 && causal != 1) return fail(TQ_EINVAL, "causal=%d (0 or 1)", causal);
  if (window < 0 || (window > 0 && !causal)) return fail(TQ_EINVAL, "window=%d (>= 0, and 0 without causal)", window);
  if ((st = check_pages(k, v)) || (st = check_batch(batch, k, &a.bt)) || (st = check_prep(prep, &a.prep))) return st;
  if (!causal && a.prep.cos_sin && !a.prep.pos) return fail(TQ_EINVAL, "a rotation without causal needs prep->pos");
  if ((st = check_handles(hk, hv, &kw, &vw)) || (st = check_cache(kw, k, "key")) || (st = check_cache(vw, v, "value"))) return st;
  if (a.prep.rot_dim > kw.d) return fail(TQ_EINVAL, "rot_dim=%d, d=%d", a.prep.rot_dim, kw.d);
  if (batch->B == 0 || batch->ntok == 0 || batch->max_q == 0) return tq_internal_ok();
  if ((st = check_rows(q, q_dtype, q_stride, Hq, kw.d, "q"))) return st;
  if (!out || !aligned(out, 16)) return fail(TQ_EINVAL, "out is NULL or misaligned (16 bytes)");
  if (!workspace || !aligned(workspace, 16)) return fail(TQ_EINVAL, "workspace is NULL or misaligned (16 bytes)");
  // The chunks' plan counts (item, key tile) pairs of one KV head in 32 bits.
  const int64_t items = batch->ntok * (Hq / Hkv) / kItemRows + std::min<int64_t>(batch->B, batch->ntok);
  const int64_t most_tiles = ((int64_t)batch->max_pages * k->page_size + kKT - 1) / kKT + kItemCost;
  if (q_dtype != TQ_F32 && flash_formats(kw, vw) && items > INT32_MAX / most_tiles)
    return fail(TQ_EUNSUPPORTED, "%lld query tiles of up to %lld key tiles: more than 2^31 pairs, split the batch", (long long)items,
                (long long)most_tiles);
  const size_t need = attn_workspace(kw, vw, a.bt, Hq, Hkv);
  if (ws_bytes < need) return fail(TQ_EINVAL, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  if (tq_internal_fault("launch")) return fail(TQ_ECUDA, "injected launch failure (TQ_FAULT=launch)");
  DeviceGuard dev(kw.device);
  if (dev.err != cudaSuccess) return fail(TQ_ECUDA, "device %d: %s", kw.device, cudaGetErrorString(dev.err));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = tq_internal_pre_launch(hk, s))) return st;
  a.q = q, a.q_stride = q_stride, a.q_dtype = q_dtype, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv;
  a.k = quant_of(kw), a.v = quant_of(vw), a.kc = view_of(kw, k), a.vc = view_of(vw, v);
  // Positions are above -2^24 and below 2^31: a window this wide is none, and what is taken off a position stays an int.
  a.scale = scale, a.causal = causal, a.window = std::min(window, 0x7e000000), a.out = out, a.err = kw.err;
  char* ws = reinterpret_cast<char*>(up(reinterpret_cast<size_t>(workspace), 256));
  const int sms = device_sms(kw.device);
  if (q_dtype != TQ_F32 && flash_formats(kw, vw)) {
    const int G = Hq / Hkv;
    const bool other = decode_formats(kw, vw, a.bt, Hkv);
    int small = 0;
    st = TQ_OK;
    if (other) {
      const DecodePlan plan = decode_plan(kw, vw, a.bt, Hq, Hkv, sms);
      small = plan.rows;
      if (G <= small) st = attn_decode_paged(a, kw, vw, plan, ws, s);
      ws += plan.total;
    }
    if (st || (int64_t)a.bt.max_q * G <= small) return st;
    const FlashPlan plan = flash_plan(kw, a.bt, Hq, Hkv, other, sms);
    return kw.d == 128 ? attn_flash<128>(a, kw, vw, plan, small, G <= small, ws, s)
                       : attn_flash<64>(a, kw, vw, plan, small, G <= small, ws, s);
  }
  return attn_simt(a, kw, vw, simt_plan(kw, vw, a.bt, Hq, Hkv, sms), ws, kw.device, s);
}

}  // extern "C"
