// wq_kv.cuh -- device pieces shared by the 4-bit KV cache kernels: where a cached row lies, and the
// value of its codes.
#pragma once
#include "wq_device.cuh"
#include "wq_internal.h"

#ifndef WQ_STATUS_ARG
#define WQ_STATUS_ARG (-1)
#endif

namespace wq {
namespace kv {

// Scale bytes of one row of D elements: q4_0 an fp16 per 32, NVFP4 an E4M3 byte per 16 (equal).
constexpr int scale_bytes(int D) { return D / 16; }

// Row (of the [pages, heads, page_size] rows) of position t >= 0 of sequence b and head h, or -1 (and
// WQ_ERR_ARG in the status word) where the position or its table entry lies outside the cache.
__device__ __forceinline__ int64_t row_of(const KvArgs& kv, int64_t b, int t, int h) {
  int64_t page = b;
  int off = t;
  bool ok = t < kv.capacity;
  if (kv.table && ok) {
    const int p = t / kv.page_size;
    off = t - p * kv.page_size;
    page = kv.table[b * kv.table_ld + p];
  }
  ok = ok && page >= 0 && page < kv.pages;
  if (!ok) {
    set_status(WQ_STATUS_ARG);
    return -1;
  }
  return (page * kv.heads + h) * (int64_t)kv.page_size + off;
}

// start[b] / counts[b] of an append or read call.
__device__ __forceinline__ int first_of(const int32_t* start, int64_t b) { return start ? start[b] : 0; }
__device__ __forceinline__ int count_of(const int32_t* counts, int64_t b, int64_t tokens) {
  return counts ? min(max(counts[b], 0), (int)tokens) : (int)tokens;
}

// The eight values of a 32-bit word of codes (element i in bits 4i .. 4i + 3).  q4_0: (c - 8) * d.
// NVFP4: (E2M1(c) * s) * g, the inner product exact.
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, float s, float g, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = (w >> (4 * i)) & 15u;
    if (FMT == WQ_Q4_0) v[i] = __fmul_rn((float)((int)c - 8), s);
    else v[i] = __fmul_rn(__fmul_rn(kE2M1[c], s), g);
  }
}
// Scale of element e of the row whose scale bytes start at p.
template <int FMT>
__device__ __forceinline__ float scale_at(const uint8_t* p, int e) {
  if (FMT == WQ_Q4_0) return f16_bits_to_f32(reinterpret_cast<const uint16_t*>(p)[e / 32]);
  return e4m3_to_f32(p[e / 16]);
}

}  // namespace kv
}  // namespace wq
