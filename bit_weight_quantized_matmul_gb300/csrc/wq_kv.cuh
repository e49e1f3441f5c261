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

__device__ __forceinline__ int page_of(const KvArgs& kv, int t) {
  return (int)(__umulhi((uint32_t)t, kv.page_mul) >> kv.page_shift);
}

// Four bytes of two E2M1 codes -> four fp16 pairs (low nibble in the low half), exact.
__device__ __forceinline__ void e2m1_pairs(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

// Four E4M3 bytes -> two fp16 pairs, exact.
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "mov.b32 {h0, h1}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h1;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

// Row (of the [pages, heads, page_size] rows) of position t of sequence b and head h, or -1 (and
// WQ_ERR_ARG in the status word) where the position or its table entry lies outside the cache.  *left: the
// tokens from t to the end of its page, whose rows follow.
__device__ __forceinline__ int64_t row_of(const KvArgs& kv, int64_t b, int64_t t, int h, int* left) {
  int64_t page = b;
  int off = (int)t;
  bool ok = t >= 0 && t < kv.capacity;
  if (kv.table && ok) {
    const int p = page_of(kv, off);
    off -= p * kv.page_size;
    page = kv.table[b * kv.table_ld + p];
  }
  ok = ok && page >= 0 && page < kv.pages;
  if (!ok) {
    set_status(WQ_STATUS_ARG);
    return -1;
  }
  *left = kv.page_size - off;
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
  if (FMT == WQ_Q4_0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn((float)((int)((w >> (4 * i)) & 15u) - 8), s);
  } else {
    uint32_t r[4];
    e2m1_pairs(w, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __fmul_rn(__fmul_rn(f16_bits_to_f32(r[i] & 0xFFFFu), s), g);
      v[2 * i + 1] = __fmul_rn(__fmul_rn(f16_bits_to_f32(r[i] >> 16), s), g);
    }
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
