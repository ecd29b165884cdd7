// Internal to libdv: what the operators over the cache (dv_append.cu,
// dv_compact.cu, dv_attention.cu) share: argument checks, the tables of the
// packed token ranges that kernels take by value, and small device helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dv_host.h"

namespace dv {

// New-token ranges of the sequences, by value in the kernel parameters.
template <int MAXB>
struct SeqTable {
  int32_t batch;
  int32_t start[MAXB];      // first new row
  int32_t pre[MAXB + 1];    // tokens before the sequence in packed buffers
};

template <int MAXB>
void fill_table(const Plan& p, SeqTable<MAXB>* t) {
  t->batch = p.B;
  for (int b = 0; b < p.B; ++b) {
    t->start[b] = p.seq_start[b];
    t->pre[b] = p.tok_pre[b];
  }
  t->pre[p.B] = p.tok_pre[p.B];
}

// The last b with pre[b] <= i (pre ascending, pre[0] = 0, i < pre[n]): the
// non-empty entry that holds i.
__device__ __forceinline__ int find_span(const int32_t* pre, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (pre[m] <= i) lo = m; else hi = m;
  }
  return lo;
}

// Two values of a 16-bit type packed in 32 bits, and back.
template <typename T>
struct Pack2;
template <>
struct Pack2<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Pack2<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// See pdl_enter in dv_kernels.cu: waits for the grids this launch depends on
// before any global memory is touched, then lets the next launch start.
__device__ __forceinline__ void ops_pdl_enter() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches `kernel` so that it may be scheduled while the stream's previous
// kernel drains (its ops_pdl_enter keeps the order).
template <typename... Params>
cudaError_t ops_launch(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                       cudaStream_t stream, const Params&... kp) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, kp...);
  return err != cudaSuccess ? err : cudaGetLastError();
}

// Validates one layer's ranges for an operator on 2-byte elements.
inline dv_status plan_layer(const dv_cache* c, int32_t layer, const int32_t* s, const int32_t* e,
                            int32_t dtype, Plan* p) {
  const dv_status st = plan_ranges(c, layer, layer < INT32_MAX ? layer + 1 : layer, s, e, p);
  if (st != DV_OK) return st;
  if (layer >= c->num_layers)
    return fail(DV_ERR_RANGE, "layer %d outside [0,%d)", layer, c->num_layers);
  if (c->elem_bytes != 2)
    return fail(DV_ERR_UNSUPPORTED, "this operator needs 2-byte elements (elem_bytes %d)",
                c->elem_bytes);
  if (dtype != DV_DTYPE_FP16 && dtype != DV_DTYPE_BF16)
    return fail(DV_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  return DV_OK;
}

// Checks the stride of a packed buffer of p.tokens rows of `heads` heads, in elements from
// row to row, and gives the bytes it spans.
inline dv_status span_rows(const Plan& p, int32_t heads, int64_t stride, const char* what,
                           size_t* span) {
  const int64_t row = (int64_t)heads * p.D;
  if (stride < row)
    return fail(DV_ERR_INVALID_ARG, "%s: a stride of %lld elements is less than a token's %lld",
                what, (long long)stride, (long long)row);
  if (stride > (int64_t)1 << 40)
    return fail(DV_ERR_INVALID_ARG, "%s: a stride of %lld elements", what, (long long)stride);
  if (stride % 8 != 0)
    return fail(DV_ERR_MISALIGNED, "%s: a stride of %lld elements is not a multiple of 8", what,
                (long long)stride);
  if (p.tokens - 1 > (((int64_t)1 << 60) - row) / stride)  // (the product below stays in range)
    return fail(DV_ERR_BUFFER_TOO_SMALL, "%s: no allocation holds %lld tokens %lld elements apart",
                what, (long long)p.tokens, (long long)stride);
  *span = (size_t)(((p.tokens - 1) * stride + row) * 2);
  return DV_OK;
}

// As resolve_cache: the cache's K and V bases, up to the last layer of the plan.
inline dv_status resolve_layers(Plan* p) {
  const int64_t dense = (int64_t)p->B * p->H * p->D * p->S;
  const size_t need = (size_t)((p->l1 - 1) * p->layer_chunks * 16 + dense * p->P);
  void* k = nullptr;
  void* v = nullptr;
  dv_status st = resolve_words(p->k, need, 16, "cache.k_base", &k);
  if (st == DV_OK) st = resolve_words(p->v, need, 16, "cache.v_base", &v);
  if (st != DV_OK) return st;
  p->k = k;
  p->v = v;
  return DV_OK;
}

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// Whether a buffer shares bytes with K or V of one of the plan's layers (not with what lies
// between them).  By address alone: the buffers need not be resolved.
inline bool overlaps_layers(const Plan& p, const void* a, size_t n) {
  const size_t bytes = (size_t)p.B * p.H * p.D * p.S * p.P;
  for (int32_t l = p.l0; l < p.l1; ++l) {
    const size_t at = (size_t)(l * p.layer_chunks) * 16;
    if (overlap(a, n, static_cast<const char*>(p.k) + at, bytes) ||
        overlap(a, n, static_cast<const char*>(p.v) + at, bytes))
      return true;
  }
  return false;
}

}  // namespace dv
