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

// c - 8 of the q4_0 codes in bits 0 .. 3 and 4 .. 7 of each half, as fp16 pairs: 1024 + c - 1032, and
// (1024 + 16 c) / 16 - 72, both exact.
__device__ __forceinline__ void signed_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"((w & 0x000F000Fu) | 0x64006400u), "r"(0xE408E408u));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(hi) : "r"((w & 0x00F000F0u) | 0x64006400u), "r"(0x2C002C00u), "r"(0xD480D480u));
}

// The eight values of a 32-bit word of codes (element i in bits 4i .. 4i + 3).  q4_0: (c - 8) * s, s its d.
// NVFP4: (E2M1(c) * E4M3) * s, the inner product exact in fp16 (pair: the block's scale in both halves), s its g.
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t pair, float s, float (&v)[8]) {
  uint32_t r[4];
  if (FMT == WQ_Q4_0) {
    signed_pairs(w, r[0], r[1]);
    signed_pairs(w >> 8, r[2], r[3]);
  } else {
    e2m1_pairs(w, r);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (FMT == WQ_NVFP4) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(pair));
    const int lo = FMT == WQ_Q4_0 ? i : 2 * i, hi = FMT == WQ_Q4_0 ? i + 4 : 2 * i + 1;
    v[lo] = __fmul_rn(f16_bits_to_f32(r[i] & 0xFFFFu), s);
    v[hi] = __fmul_rn(f16_bits_to_f32(r[i] >> 16), s);
  }
}
// The scale bits of element e of the row whose scale bytes start at p.
template <int FMT>
__device__ __forceinline__ uint32_t scale_at(const uint8_t* p, int e) {
  return FMT == WQ_Q4_0 ? reinterpret_cast<const uint16_t*>(p)[e / 32] : p[e / 16];
}
// An E4M3 byte as an fp16 pair of equals.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(b * 0x0101u));
  return r;
}

// ---- what a row of the SEL attention kernels sees, as bits
// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }
// Of the 32 tokens from t0 on: those in [lo, hi), the first `sinks` below hi, and, where bits of drafted nodes are given
// (`words` of them), of the positions base + j below `end` those whose bit j is set.  hi is at most base then.
// JUMP: a branch around the nodes, else none, so that the loads of several calls are under way together.
template <bool JUMP>
__device__ __forceinline__ uint32_t sight(int t0, int lo, int hi, int sinks, const uint32_t* nodes, int words, int base, int end) {
  const uint32_t see = (bits_below(hi - t0) & ~bits_below(lo - t0)) | bits_below(min(sinks, hi) - t0);
  const bool some = nodes && end > t0 && base < t0 + 32;
  if (JUMP && !some) return see;
  const int at = some ? t0 - base : 0, w = at >> 5;      // bit of t0, -31 or more
  const uint32_t a = some && w >= 0 && w < words ? nodes[w] : 0u, b = some && w + 1 < words ? nodes[w + 1] : 0u;
  return see | (__funnelshift_r(a, b, at & 31) & (some ? bits_below(end - t0) : 0u));
}

// Which sequence sees the rank'th most tokens (of equals the lower number first): where there are more blocks than places, those
// with the most to do begin first.  64 sequences of 8 heads behind a window of 4096 are 512 blocks for 456 places: the last 56
// began after 23 .. 42 us of 87, most of them as long as any.  Lengths are on the device, so the host cannot order them.
// batch <= kSorted; all threads of the block; room: batch ints and one in shared memory.
constexpr int kSorted = 256;
template <int THREADS>
__device__ __forceinline__ int64_t by_length(const AttendArgs& a, int rank, int* room) {
  const int batch = (int)a.batch;
  for (int b = threadIdx.x; b < batch; b += THREADS) {
    const int n = count_of(a.counts, b, a.tokens), len = max(a.lens[b], 0), held = (int)min((int64_t)len, a.kv.capacity);
    const int lo = a.window ? (int)min((int64_t)held, max((int64_t)0, (int64_t)len - n - a.window + 1)) : 0;
    room[b] = n > 0 ? held - lo + (a.window ? min(a.sinks, lo) : 0) : 0;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < batch; b += THREADS) {
    const int mine = room[b];
    int before = 0;
    for (int c = 0; c < batch; ++c) {
      const int other = room[c];
      before += other > mine || (other == mine && c < b);
    }
    if (before == rank) room[batch] = b;
  }
  __syncthreads();
  const int b = room[batch];
  __syncthreads();                                 // `room` is free again
  return b;
}

// ---- arithmetic of the attention kernels
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The top bit of each half of an fp16 pair that is 8192 or more in magnitude (or no finite number).
__device__ __forceinline__ uint32_t large(uint32_t x) { return ((x & 0x70007000u) + 0x10001000u) & 0x80008000u; }

}  // namespace kv
}  // namespace wq
