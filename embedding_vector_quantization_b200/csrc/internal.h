// Library-internal helpers shared between translation units (not part of the ABI).
#pragma once

// Records `fmt` as this thread's tq_last_error() message and returns `code`.
__attribute__((visibility("hidden"))) int tq_internal_fail(int code, const char* fmt, ...);

#include <stddef.h>
#include <stdint.h>
struct tq_handle;
// Workspace bytes tq_attn_decode needs at least (tq_attn_workspace_bytes may ask for more: the
// scores buffer of the two-kernel attention, used only when the workspace holds it).
extern "C" __attribute__((visibility("hidden"))) size_t tq_internal_attn_workspace_min_bytes(
    const tq_handle* hk, const tq_handle* hv, int B, int Hq, int Hkv, int64_t L_cap);

#include <cuda_runtime.h>

// What the other translation units may know of a handle (device pointers stay the handle's).
struct tq_view {
  int d, bits, m, norm_dtype, codes_B, signs_B, device, polar;
  const float *PiT, *Pi, *MT, *ST, *S, *cent, *bnd;   // fp32: [d][d], [d][d], [d][m], [d][m], [m][d], centroids, boundaries
  const double* t64;       // d <= 256: Pi [d][d], S [m][d], M [m][d], 16 boundaries (+inf padded), 16 centroids
  // d = 64 or 128 (m = 0 or d): f16 operands of the paged expansion, for keys and for values (tq_api.cu); NULL otherwise
  const uint8_t *ops16k, *ops16v;
  const uint8_t* ops_app;  // d = 64 or 128 (m = 0 or d), with codes: f16 pairs of Pi and M (tq_api.cu); NULL otherwise
  float m_abs, m_norm;     // largest row of M in the 1-norm and the 2-norm
  float cent_up;           // the factor in [1, 2) with which the centroids come nearest to f16 (table_factor in tq_api.cu)
  int* err;                // device error word
};
__attribute__((visibility("hidden"))) void tq_internal_view(const tq_handle* h, tq_view* v);
__attribute__((visibility("hidden"))) int tq_internal_ok();
__attribute__((visibility("hidden"))) bool tq_internal_fault(const char* what);
// TQ_FAULT=timeout for a call on h (no lengths to check).
__attribute__((visibility("hidden"))) int tq_internal_pre_launch(const tq_handle* h, cudaStream_t s);
// Brackets one kernel launch with timer events while the timer is on (KernelScope of tq_api.cu).
struct tq_launch_scope {
  void* impl;
  __attribute__((visibility("hidden"))) tq_launch_scope(const char* name, cudaStream_t s);
  __attribute__((visibility("hidden"))) ~tq_launch_scope();
};
