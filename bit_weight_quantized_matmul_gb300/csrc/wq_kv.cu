// wq_kv.cu -- quantising rows into the 4-bit KV cache as they are written, and reading them back.
//
// Both move each element once; HBM bounds them (append: 2 bytes in, 9/16 out; read the other way
// round), and the launch a call of few tokens.  A thread owns the same eight elements of a head in up to
// kUnroll tokens of one sequence, whose loads are in flight together: one 16-byte access on the bf16 side,
// four bytes of codes.  A q4_0 block is then four neighbouring lanes, an NVFP4 block two, and the
// block's scale a maximum over them.
#include <cuda_runtime.h>

#include "wq_kv.cuh"

namespace wq {
namespace {

// Small blocks and many of them beat large ones: 16 x 1500 tokens of 20 heads of 64 (q4_0) are appended in 47 us
// (3.3 TB/s of 6.8 for a copy) and read in 31 (5.0 TB/s); blocks of 256 at 64 registers appended in 53, and read
// in 52 where the small ones, with the decode of that time, took 37.
constexpr int kThreads = 128, kUnroll = 4, kMinBlocks = 12;
// NVFP4's divisions need the registers (4 x 2048 tokens of 8 heads of 128: 12.3 us, 12.8 at 12 blocks).
constexpr int append_blocks(int fmt) { return fmt == WQ_Q4_0 ? 12 : 8; }

__device__ __forceinline__ void widen8(const uint32_t (&u)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// d of a q4_0 block, four lanes holding its 32 bf16 values: the signed value of largest magnitude, the
// first of equals, over -8, as fp16 bits.  As 16-bit integers the positive values order by magnitude, and
// so do the negative ones with the sign bit flipped: two maxima P and N, which differ unless +a and -a are
// both there; then the first of them decides.  A NaN's magnitude is the largest, so a NaN makes d a NaN
// and the block reads back as NaN.
__device__ __forceinline__ uint16_t q4_0_d(const uint32_t (&u)[4], int lane) {
  uint32_t p = u[0], n = u[0] ^ 0x80008000u;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    p = __vmaxs2(p, u[i]);
    n = __vmaxs2(n, u[i] ^ 0x80008000u);
  }
  uint32_t m = __vmaxs2(__byte_perm(p, n, 0x5410), __byte_perm(p, n, 0x7632));   // P low, N high
  m = __vmaxs2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = __vmaxs2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
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
// a half-integer exactly or at least 2^-12 away from one; x RN(1 / d), off by 2^-20 at most, rounded to a
// multiple of 2^-13 (the addition of 1536 does it) is on the same side of every half-integer and on it where
// x / d is.  Adding up to 12582912 + 8 then rounds to an integer, ties to even, whose low bits are the code.
__device__ __forceinline__ uint32_t q4_0_codes(const uint32_t (&u)[4], uint16_t d_bits) {
  const float d = f16_bits_to_f32(d_bits);
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

// x / s rounded to nearest even for eight x sharing one s: Markstein's division (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990): with
// y = RN(1 / s), q = RN(x y) and the exact residual r = x - q s, RN(q + r y) is RN(x / s) while nothing
// leaves the normal range.  s outside [2^-100, 2^100] takes the plain division.  Quotients past 16 in
// magnitude, which every code saturates, come back as q, a zero or subnormal x as a zero of its sign.
__device__ __forceinline__ void divide8(const float (&x)[8], float s, float (&q)[8]) {
  const float m = fabsf(s);
  if (m > 7.888609e-31f && m < 1.2676506e30f) {
    const float y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q0 = __fmul_rn(x[i], y);
      const float q1 = __fmaf_rn(__fmaf_rn(-q0, s, x[i]), y, q0);
      q[i] = fabsf(q0) <= 16.0f ? q1 : q0;
    }
  } else {
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
  const float S = __fmul_rn(e4m3_to_f32(s), g);
  if (S == 0.0f) return 0u;  // a block whose scale underflows keeps codes 0
  divide8(x, S, q);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = copysignf(q[i], x[i]);   // a negative that rounds to zero stays negative
  return f32x8_to_e2m1x8(q);
}

// Rows of a thread's tokens: looked up once per page, counted on from the first token's row within it.
struct Rows {
  int64_t first = -1;
  int left = 0;         // tokens from the first one to the end of its page
  __device__ __forceinline__ int64_t at(const KvArgs& kv, int64_t b, int64_t t, int h, int ahead) {
    if (ahead < left) return first + ahead;
    int rest;
    const int64_t row = kv::row_of(kv, b, t, h, &rest);
    if (ahead == 0 && row >= 0) {
      first = row;
      left = rest;
    }
    return row;
  }
};

// A block covers one head of K (blockIdx.y 0) or V in kUnroll rounds of `wide` neighbouring tokens of one
// sequence (blockIdx.z): blockIdx.x counts heads within chunks of tokens, so that neighbouring blocks
// read or write neighbouring bf16 rows, and a block's codes are contiguous within a page.
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, append_blocks(FMT)) kv_append_kernel(const __grid_constant__ KvMoveArgs a, const int wide) {
  constexpr int kPer = D / 8;           // threads a token
  const int which = blockIdx.y, chunk = blockIdx.x / (unsigned)a.kv.heads, h = blockIdx.x - chunk * a.kv.heads;
  const int tok = threadIdx.x / kPer, e = (threadIdx.x % kPer) * 8, i0 = chunk * wide * kUnroll;
  for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const int n = kv::count_of(a.counts, b, a.tokens);
    if (i0 >= n) continue;
    const int64_t start = kv::first_of(a.start, b);
    const float g = FMT == WQ_NVFP4 && a.kv.g[which] ? *a.kv.g[which] : 1.0f;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(a.x[which].p) + b * a.x[which].batch + h * a.x[which].head + e;
    uint4 u[kUnroll];
    int64_t row[kUnroll];
    Rows rows;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * wide + tok;
      const bool in = tok < wide && i < n;
      u[k] = in ? *reinterpret_cast<const uint4*>(src + i * a.x[which].token) : make_uint4(0, 0, 0, 0);
      row[k] = in ? rows.at(a.kv, b, start + i, h, k * wide) : -1;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (i0 + k * wide >= n) break;      // for the whole block: its lanes exchange values below
      const uint32_t v[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      uint32_t w;
      uint16_t d = 0;
      uint8_t sb = 0;
      if (FMT == WQ_Q4_0) {
        d = q4_0_d(v, threadIdx.x & 31);
        w = q4_0_codes(v, d);
      } else {
        w = encode_nvfp4(v, g, sb);
      }
      if (row[k] >= 0) {
        if (FMT == WQ_Q4_0) {
          if ((e & 31) == 0) reinterpret_cast<uint16_t*>(a.kv.scales[which])[row[k] * (D / 32) + e / 32] = d;
        } else {
          if ((e & 15) == 0) a.kv.scales[which][row[k] * (D / 16) + e / 16] = sb;
        }
        *reinterpret_cast<uint32_t*>(a.kv.codes[which] + row[k] * (D / 2) + e / 2) = w;
      }
    }
  }
}

template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(kThreads, kMinBlocks) kv_read_kernel(const __grid_constant__ KvMoveArgs a, const int wide) {
  constexpr int kPer = D / 8;
  const int which = a.x[0].p ? blockIdx.y : 1, chunk = blockIdx.x / (unsigned)a.kv.heads, h = blockIdx.x - chunk * a.kv.heads;
  const int tok = threadIdx.x / kPer, e = (threadIdx.x % kPer) * 8, i0 = chunk * wide * kUnroll;
  if (tok >= wide) return;
  for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const int n = kv::count_of(a.counts, b, a.tokens);
    const int64_t start = kv::first_of(a.start, b);
    const float g = FMT == WQ_NVFP4 && a.kv.g[which] ? *a.kv.g[which] : 1.0f;
    const int64_t base = b * a.x[which].batch + h * a.x[which].head + e;
    uint32_t w[kUnroll], sc[kUnroll];
    Rows rows;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * wide + tok;
      w[k] = FMT == WQ_Q4_0 ? 0x88888888u : 0u;    // a row that is not there reads as zero
      sc[k] = 0u;
      const int64_t row = i < n ? rows.at(a.kv, b, start + i, h, k * wide) : -1;
      if (row >= 0) {
        w[k] = *reinterpret_cast<const uint32_t*>(a.kv.codes[which] + row * (D / 2) + e / 2);
        sc[k] = kv::scale_at<FMT>(a.kv.scales[which] + row * kv::scale_bytes(D), e);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * wide + tok;
      if (i >= a.tokens) break;
      float v[8];
      if (FMT == WQ_Q4_0) kv::decode8<FMT>(w[k], 0u, f16_bits_to_f32(sc[k]), v);
      else kv::decode8<FMT>(w[k], kv::e4m3_pair(sc[k]), g, v);
      const int64_t at = base + i * a.x[which].token;
      if (F32) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.x[which].p) + at);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.x[which].p) + at) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      }
    }
  }
}

// Few tokens take a block of as few warps.
struct Grid {
  int wide;
  dim3 blocks, threads;
  bool ok;
};
Grid grid_for(const KvMoveArgs& a, int sides) {
  Grid g{};
  const int per = a.kv.dim / 8;
  g.wide = (int)(a.tokens < kThreads / per ? a.tokens : kThreads / per);
  g.threads = dim3((unsigned)((g.wide * per + 31) / 32 * 32));
  const int64_t chunks = (a.tokens + g.wide * kUnroll - 1) / (g.wide * kUnroll);
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
  const Grid g = grid_for(a, 2);
  if (!g.ok) return WQ_ERR_SHAPE;
  kv_append_kernel<FMT, D><<<g.blocks, g.threads, 0, s>>>(a, g.wide);
  return launched();
}
template <int FMT, int D>
int read_t(const KvMoveArgs& a, cudaStream_t s) {
  const Grid g = grid_for(a, (a.x[0].p ? 1 : 0) + (a.x[1].p ? 1 : 0));
  if (!g.ok) return WQ_ERR_SHAPE;
  if (a.f32) kv_read_kernel<FMT, D, true><<<g.blocks, g.threads, 0, s>>>(a, g.wide);
  else kv_read_kernel<FMT, D, false><<<g.blocks, g.threads, 0, s>>>(a, g.wide);
  return launched();
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
