// wq_kv.cu -- quantising rows into the 4-bit KV cache as they are written, and reading them back.
//
// Both move each element once (append: 2 bytes in, 9/16 out; read the other way round).  HBM bounds the reading (8 x
// 12000 .. 16384 tokens of 8 heads of 128, NVFP4, to bf16: 103 us, 6.5 TB/s of 6.8 for a copy), instruction issue the
// appending (16 x 1500 x 20 x 64, q4_0: 35 us, 4.5 TB/s; 132 instructions per eight elements, issued 85 % of the
// time; 4 x 333 .. 2048 x 8 x 128, NVFP4: 10 us, at 8 blocks an SM, half of its warps there, issuing 65 % of the time
// and waiting for the loads at the block's beginning), the launch a call of few tokens.  A thread owns the same eight elements of a head in up to
// eight tokens of one sequence, whose loads are in flight together: one 16-byte access on the bf16 side,
// four bytes of codes.  A q4_0 block is then four neighbouring lanes, an NVFP4 block two, and the
// block's scale a maximum over them.
#include <cuda_runtime.h>

#include "wq_kv.cuh"

namespace wq {
namespace {

// Small blocks and many of them, of as many rounds as their registers hold: each round's loads are in flight
// together, and a block's beginning costs as much as two rounds.  8 x 1700 .. 2000 tokens of 20 heads of 64 in pages
// of 64 (q4_0) are appended in 24 us (4.0 TB/s) and read in 18 (5.3); with 2 rounds in 30 and 26, with 8 and 4 in 35
// and 19; at 8 blocks an SM in 26 and 21.
constexpr int kThreads = 128, kAppendRounds = 4, kReadRounds = 8, kReadRoundsFew = 2;
constexpr int kMinBlocks = 12, kSms = 152;
// NVFP4's divisions need the registers (4 x 2048 tokens of 8 heads of 128: 12.3 us, 12.8 at 12 blocks).
constexpr int append_blocks(int fmt) { return fmt == WQ_Q4_0 ? 12 : 8; }

__device__ __forceinline__ void widen8(const uint32_t (&u)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t max_s2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_u2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_u2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Pairs of fp32, one instruction for both.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(float x) { return pair(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ void unpair(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_p(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_p(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_p(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// d of a q4_0 block, four lanes holding its 32 bf16 values: the signed value of largest magnitude, the
// first of equals, over -8, as fp16 bits.  As signed 16-bit integers the positive values order by magnitude,
// as unsigned ones the negative do: two maxima P and N, which differ in magnitude unless +a and -a are both
// there; then the first of them decides.  A NaN's magnitude is the largest, so a NaN makes d a NaN and the
// block reads back as NaN.
__device__ __forceinline__ uint16_t q4_0_d(const uint32_t (&u)[4], int lane) {
  const uint32_t p = max_s2(max_s2(u[0], u[1]), max_s2(u[2], u[3]));
  const uint32_t n = max_u2(max_u2(u[0], u[1]), max_u2(u[2], u[3])) ^ 0x80008000u;
  uint32_t m = max_s2(__byte_perm(p, n, 0x5410), __byte_perm(p, n, 0x7632));   // P low, N high
  m = max_s2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max_s2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const int pos = (int16_t)(m & 0xFFFFu), neg = (int16_t)(m >> 16);
  bool minus = neg > pos;
  if (__any_sync(0xFFFFFFFFu, neg == pos)) {     // rare: the lower index of the two magnitudes
    uint32_t first = 64;                         // 2 * index + sign
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      const uint32_t b = (u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
      if ((int)(b & 0x7FFFu) == pos) first = 2 * (8 * (lane & 3) + i) + (b >> 15);
    }
    first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 1));
    first = min(first, __shfl_xor_sync(0xFFFFFFFFu, first, 2));
    if (neg == pos) minus = (first & 1u) != 0;
  }
  const float ext = __uint_as_float((uint32_t)(minus ? neg | 0x8000 : pos) << 16);
  return __half_as_ushort(__float2half_rn(__fmul_rn(ext, -0.125f)));   // exact but for the fp16 rounding
}

// Codes clamp(rint(x / d) + 8, 0, 15) of eight bf16 values.  x has 8 significant bits and d 11, so x / d is
// a half-integer exactly or at least 2^-12 away from one; x times 1 / d to an ulp, off by 2^-19 at most, rounded to
// a multiple of 2^-13 (the addition of 1536 does it) is on the same side of every half-integer and on it where
// x / d is.  Adding up to 12582912 + 8 then rounds to an integer, ties to even, whose low bits are the code.
// With d a normal fp16 number |x / d| <= 8 (1 + 2^-11), so only 16 has to be clamped.
__device__ __forceinline__ uint32_t q4_0_codes(const uint32_t (&u)[4], uint16_t d_bits) {
  const float d = f16_bits_to_f32(d_bits);
  const uint32_t e = d_bits & 0x7C00u;
  if (e != 0 && e != 0x7C00u) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
    const uint64_t yy = pair(y), round = pair(1536.0f), code = pair(12581384.0f);
    uint32_t c[4];                                 // codes of elements i and i + 4 in its halves
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = u[i >> 1], b = u[2 + (i >> 1)];
      uint32_t lo, hi;
      unpair(add_p(fma_p(pair(i & 1 ? a & 0xFFFF0000u : a << 16, i & 1 ? b & 0xFFFF0000u : b << 16), yy, round), code), lo, hi);
      c[i] = min_u2(__byte_perm(lo, hi, 0x5410), 0x000F000Fu);
    }
    return (c[0] + c[1] * 16u) + (c[2] + c[3] * 16u) * 256u;
  }
  if (d == 0.0f) return 0x88888888u;               // every code stands for zero
  float x[8];
  widen8(u, x);
  const float y = __frcp_rn(d);
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float t = fminf(fmaxf(__fmaf_rn(x[i], y, 1536.0f), 1528.0f), 1543.0f);
    w = w * 16u + __float_as_uint(__fadd_rn(t, 12581384.0f));
  }
  return w - 0x4B400000u * 0x11111111u;            // 0x4B400000: the bits of 12582912
}

// x / s rounded to nearest even for eight x sharing one s, none larger than amax in magnitude: Markstein's
// division (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J.
// Res. Dev. 34(1), 1990): with y = RN(1 / s), q = RN(x y) and the exact residual r = x - q s, RN(q + r y) is
// RN(x / s) while nothing leaves the normal range.  Quotients past 16 in magnitude (which every code saturates) and
// s outside [2^-100, 2^100] take the plain division; a zero or subnormal x comes back as a zero.
__device__ __forceinline__ void divide8(const uint32_t (&u)[4], float amax, float s, float (&q)[8]) {
  const float m = fabsf(s);
  if (m > 7.888609e-31f && m < 1.2676506e30f && amax <= 16.0f * m) {
    const float y = __frcp_rn(s);
    const uint64_t yy = pair(y), ss = pair(-s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = pair(u[i] << 16, u[i] & 0xFFFF0000u), q0 = mul_p(x, yy);
      uint32_t lo, hi;
      unpair(fma_p(fma_p(q0, ss, x), yy, q0), lo, hi);
      q[2 * i] = __uint_as_float(lo);
      q[2 * i + 1] = __uint_as_float(hi);
    }
  } else {
    float x[8];
    widen8(u, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], s);
  }
}

// Codes of eight bf16 values of an NVFP4 block (two lanes hold its 16) and its E4M3 scale.
__device__ __forceinline__ uint32_t encode_nvfp4(const uint32_t (&u)[4], float g, uint8_t& s_byte) {
  float x[8], q[8], amax = 0.0f;
  widen8(u, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  const uint32_t s = f32_to_e4m3_cvt(__fdiv_rn(__fdiv_rn(amax, 6.0f), g));
  s_byte = (uint8_t)s;
  const float S = __fmul_rn(f16_bits_to_f32(kv::e4m3_pair(s) & 0xFFFFu), g);
  if (!(fabsf(S) > 0.0f)) return 0u;  // a block whose scale underflows keeps codes 0
  divide8(u, amax, S, q);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = copysignf(q[i], x[i]);   // a negative that rounds to zero stays negative
  return f32x8_to_e2m1x8(q);
}

// Codes of eight values and their block's scale bits; all lanes of a warp together.
template <int FMT>
__device__ __forceinline__ uint32_t encode8(const uint4& x, float g, uint32_t& scale) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  if (FMT == WQ_Q4_0) {
    const uint16_t d = q4_0_d(u, threadIdx.x & 31);
    scale = d;
    return q4_0_codes(u, d);
  }
  uint8_t s;
  const uint32_t w = encode_nvfp4(u, g, s);
  scale = s;
  return w;
}
template <int FMT>
__device__ __forceinline__ void store_scale(uint8_t* row, int e, uint32_t scale) {
  if (FMT == WQ_Q4_0) {
    if ((e & 31) == 0) reinterpret_cast<uint16_t*>(row)[e / 32] = (uint16_t)scale;
  } else {
    if ((e & 15) == 0) row[e / 16] = (uint8_t)scale;
  }
}

// A block covers one head of K (blockIdx.y 0) or V in some rounds of `wide` neighbouring tokens of one
// sequence (blockIdx.z): blockIdx.x counts heads within chunks of tokens, so that neighbouring blocks
// read or write neighbouring bf16 rows, and a block's codes are contiguous within a page.  The chunks
// begin at positions that are multiples of their length, so that a round (8 or 16 tokens; a page's are a multiple of
// 16) of a whole block never leaves its page: the block looks up one row a round, or one in all.  Blocks at the ends, and calls of few tokens, look up
// each token.  (16 x 1500 tokens of 20 heads of 64 in one slab each: a look-up per token took 42 us to append and
// 31 to read, one per block 34 and 23.)
template <int D, int ROUNDS>
struct Split {
  static constexpr int kPer = D / 8, kWide = kThreads / kPer, kSpan = kWide * ROUNDS;   // threads a token; tokens a round, a block
  // Tokens by which the first chunk begins before the call's first.
  static __device__ __forceinline__ int lead(const KvMoveArgs& a, int wide, int64_t start) {
    return wide == kWide ? (int)(start & (kSpan - 1)) : 0;
  }
};
// Row of the token at position t, or -1 with the status set.
__device__ __forceinline__ int64_t row_at(const KvMoveArgs& a, int64_t b, int64_t t, int h) {
  int left;
  return kv::row_of(a.kv, b, t, h, &left);
}
// Where the codes and the scales of eight elements lie: of row `row`, element e.
template <int D>
struct Place {
  uint8_t *codes, *scales;
  __device__ __forceinline__ Place(const KvArgs& kv, int which, int64_t row, int e)
      : codes(kv.codes[which] + row * (D / 2) + e / 2), scales(kv.scales[which] + row * kv::scale_bytes(D)) {}
  __device__ __forceinline__ Place(uint8_t* c, uint8_t* s) : codes(c), scales(s) {}
  __device__ __forceinline__ Place ahead(int rows) const { return Place(codes + rows * (D / 2), scales + rows * kv::scale_bytes(D)); }
};

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, append_blocks(FMT)) kv_append_kernel(const __grid_constant__ KvMoveArgs a, const int wide) {
  constexpr int kPer = Split<D, kAppendRounds>::kPer, kWide = Split<D, kAppendRounds>::kWide, kSpan = Split<D, kAppendRounds>::kSpan;
  const int which = blockIdx.y, chunk = blockIdx.x / (unsigned)a.kv.heads, h = blockIdx.x - chunk * a.kv.heads;
  const int tok = threadIdx.x / kPer, e = (threadIdx.x % kPer) * 8;
  for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const int64_t start = kv::first_of(a.start, b), step = a.x[which].token;
    const int64_t i0 = (int64_t)chunk * (wide * kAppendRounds) - Split<D, kAppendRounds>::lead(a, wide, start);
    const int64_t rest = kv::count_of(a.counts, b, a.tokens) - i0;   // tokens from i0 on
    if (rest <= 0) continue;
    const float g = FMT == WQ_NVFP4 && a.kv.g[which] ? *a.kv.g[which] : 1.0f;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(a.x[which].p) + b * a.x[which].batch + h * a.x[which].head +
                          (i0 + tok) * step + e;
    uint4 u[kAppendRounds];
    const auto store = [&](int k, bool there, Place<D> p) {     // all lanes
      uint32_t sc;
      const uint32_t w = encode8<FMT>(u[k], g, sc);
      if (!there) return;
      *reinterpret_cast<uint32_t*>(p.codes) = w;
      store_scale<FMT>(p.scales, e, sc);
    };
    if (wide == kWide && i0 >= 0 && rest >= kSpan) {
#pragma unroll
      for (int k = 0; k < kAppendRounds; ++k) u[k] = *reinterpret_cast<const uint4*>(src + k * kWide * step);
      int left;
      const int64_t row = kv::row_of(a.kv, b, start + i0, h, &left);
      if (row >= 0 && left >= kSpan) {
        const Place<D> first(a.kv, which, row + tok, e);
#pragma unroll
        for (int k = 0; k < kAppendRounds; ++k) store(k, true, first.ahead(k * kWide));
      } else {
        const int64_t mine = row_at(a, b, start + i0 + (threadIdx.x % kAppendRounds) * kWide, h);   // lane k: round k's
#pragma unroll
        for (int k = 0; k < kAppendRounds; ++k) {
          const int64_t r = __shfl_sync(0xFFFFFFFFu, mine, k);
          store(k, r >= 0, Place<D>(a.kv, which, r + tok, e));
        }
      }
      continue;
    }
    const auto in = [&](int k) { return tok < wide && i0 + k * wide + tok >= 0 && k * wide + tok < rest; };
#pragma unroll
    for (int k = 0; k < kAppendRounds; ++k) u[k] = in(k) ? *reinterpret_cast<const uint4*>(src + k * wide * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kAppendRounds; ++k) {
      if (k * wide >= rest) break;       // for the whole block: its lanes exchange values
      const int64_t row = in(k) ? row_at(a, b, start + i0 + k * wide + tok, h) : -1;
      store(k, row >= 0, Place<D>(a.kv, which, row, e));
    }
  }
}

template <int FMT, bool F32>
__device__ __forceinline__ void put8(void* p, int64_t at, uint32_t w, uint32_t sc, float g) {
  float v[8];
  if (FMT == WQ_Q4_0) kv::decode8<FMT>(w, 0u, f16_bits_to_f32(sc), v);
  else kv::decode8<FMT>(w, kv::e4m3_pair(sc), g, v);
  if (F32) {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

template <int FMT, int D, bool F32, int ROUNDS>
__global__ void __launch_bounds__(kThreads, kMinBlocks) kv_read_kernel(const __grid_constant__ KvMoveArgs a, const int wide) {
  constexpr int kPer = Split<D, ROUNDS>::kPer, kWide = Split<D, ROUNDS>::kWide, kSpan = Split<D, ROUNDS>::kSpan;
  const int which = a.x[0].p ? blockIdx.y : 1, chunk = blockIdx.x / (unsigned)a.kv.heads, h = blockIdx.x - chunk * a.kv.heads;
  const int tok = threadIdx.x / kPer, e = (threadIdx.x % kPer) * 8;
  if (tok >= wide) return;
  for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const int64_t start = kv::first_of(a.start, b), step = a.x[which].token;
    const int64_t i0 = (int64_t)chunk * (wide * ROUNDS) - Split<D, ROUNDS>::lead(a, wide, start);
    const int64_t rest = kv::count_of(a.counts, b, a.tokens) - i0;   // held tokens from i0 on
    const float g = FMT == WQ_NVFP4 && a.kv.g[which] ? *a.kv.g[which] : 1.0f;
    const int64_t at = b * a.x[which].batch + h * a.x[which].head + (i0 + tok) * step + e;
    uint32_t w[ROUNDS], sc[ROUNDS];
    const auto load = [&](int k, bool there, Place<D> p) {
      w[k] = FMT == WQ_Q4_0 ? 0x88888888u : 0u;    // a row that is not there reads as zero
      sc[k] = 0u;
      if (!there) return;
      w[k] = *reinterpret_cast<const uint32_t*>(p.codes);
      sc[k] = kv::scale_at<FMT>(p.scales, e);
    };
    if (wide == kWide && i0 >= 0 && rest >= kSpan) {
      int left;
      const int64_t row = kv::row_of(a.kv, b, start + i0, h, &left);
      if (row >= 0 && left >= kSpan) {
        const Place<D> first(a.kv, which, row + tok, e);
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) load(k, true, first.ahead(k * kWide));
      } else {
        const int64_t mine = row_at(a, b, start + i0 + (threadIdx.x % ROUNDS) * kWide, h);   // lane k: round k's
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
          const int64_t r = __shfl_sync(0xFFFFFFFFu, mine, k);
          load(k, r >= 0, Place<D>(a.kv, which, r + tok, e));
        }
      }
#pragma unroll
      for (int k = 0; k < ROUNDS; ++k) put8<FMT, F32>(a.x[which].p, at + k * kWide * step, w[k], sc[k], g);
      continue;
    }
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      const int i = k * wide + tok;
      const int64_t row = i0 + i >= 0 && i < rest ? row_at(a, b, start + i0 + i, h) : -1;
      load(k, row >= 0, Place<D>(a.kv, which, row, e));
    }
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      const int64_t i = i0 + k * wide + tok;
      if (i >= 0 && i < a.tokens) put8<FMT, F32>(a.x[which].p, at + k * wide * step, w[k], sc[k], g);
    }
  }
}

// Few tokens take a block of as few warps.
struct Grid {
  int wide;
  dim3 blocks, threads;
  bool ok;
};
Grid grid_for(const KvMoveArgs& a, int sides, int rounds) {
  Grid g{};
  const int per = a.kv.dim / 8;
  g.wide = (int)(a.tokens < kThreads / per ? a.tokens : kThreads / per);
  g.threads = dim3((unsigned)((g.wide * per + 31) / 32 * 32));
  const int64_t span = g.wide * rounds, lead = g.wide == kThreads / per && a.start ? span - 1 : 0;
  const int64_t chunks = (a.tokens + lead + span - 1) / span;
  g.ok = chunks * a.kv.heads <= 0x7FFFFFFF;
  g.blocks = dim3((unsigned)(chunks * a.kv.heads), (unsigned)sides, (unsigned)(a.batch < 65535 ? a.batch : 65535));
  return g;
}

int launched() {
  count_launch();
  return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

template <int FMT, int D>
int append_t(const KvMoveArgs& a, cudaStream_t s) {
  const Grid g = grid_for(a, 2, kAppendRounds);
  if (!g.ok) return WQ_ERR_SHAPE;
  kv_append_kernel<FMT, D><<<g.blocks, g.threads, 0, s>>>(a, g.wide);
  return launched();
}
template <int FMT, int D, int ROUNDS>
int read_t(const KvMoveArgs& a, const Grid& g, cudaStream_t s) {
  if (!g.ok) return WQ_ERR_SHAPE;
  if (a.f32) kv_read_kernel<FMT, D, true, ROUNDS><<<g.blocks, g.threads, 0, s>>>(a, g.wide);
  else kv_read_kernel<FMT, D, false, ROUNDS><<<g.blocks, g.threads, 0, s>>>(a, g.wide);
  return launched();
}
// Fewer rounds a block where eight would leave half of the device's places empty: 3 x 777 tokens of 8 heads of 128 in
// pages of 16 to fp32 take 8.0 us with eight rounds (624 blocks), 6.3 with two, 100 tokens 3.3 and 2.3; 2 x 2500 of 20
// heads of 64 (1600 blocks) 6.1 and 8.9.
template <int FMT, int D>
int read_t(const KvMoveArgs& a, cudaStream_t s) {
  const int sides = (a.x[0].p ? 1 : 0) + (a.x[1].p ? 1 : 0);
  const Grid g = grid_for(a, sides, kReadRounds);
  if ((int64_t)g.blocks.x * g.blocks.y * g.blocks.z >= kSms * kMinBlocks / 2) return read_t<FMT, D, kReadRounds>(a, g, s);
  return read_t<FMT, D, kReadRoundsFew>(a, grid_for(a, sides, kReadRoundsFew), s);
}

}  // namespace

int kv_append(const KvMoveArgs& a, cudaStream_t s) {
  if (a.kv.fmt == WQ_Q4_0) return a.kv.dim == 64 ? append_t<WQ_Q4_0, 64>(a, s) : append_t<WQ_Q4_0, 128>(a, s);
  return a.kv.dim == 64 ? append_t<WQ_NVFP4, 64>(a, s) : append_t<WQ_NVFP4, 128>(a, s);
}

int kv_read(const KvMoveArgs& a, cudaStream_t s) {
  if (a.kv.fmt == WQ_Q4_0) return a.kv.dim == 64 ? read_t<WQ_Q4_0, 64>(a, s) : read_t<WQ_Q4_0, 128>(a, s);
  return a.kv.dim == 64 ? read_t<WQ_NVFP4, 64>(a, s) : read_t<WQ_NVFP4, 128>(a, s);
}

int take_status_kv() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
