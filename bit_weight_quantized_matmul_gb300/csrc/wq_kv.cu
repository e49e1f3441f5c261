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

constexpr int kThreads = 512;
constexpr int kUnroll = 4;

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

__device__ __forceinline__ void widen8(const uint32_t (&u)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_bits_to_f32(u[i] & 0xFFFFu);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Codes of eight bf16 values of a q4_0 block (four lanes hold its 32) and its d: the signed value of
// largest magnitude, the first of equals, over -8.  The key orders by magnitude, then lower index; a
// NaN's magnitude bits are the largest, so a NaN makes d a NaN and the block reads back as NaN.
__device__ __forceinline__ uint32_t encode_q4_0(const uint32_t (&u)[4], int lane, uint16_t& d_bits) {
  uint32_t key = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = (u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    const uint32_t idx = 8 * (lane & 3) + i;
    key = max(key, ((b & 0x7FFFu) << 6) | ((31u - idx) << 1) | (b >> 15));
  }
  key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, 1));
  key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, 2));
  const float ext = bf16_bits_to_f32((key >> 6) | ((key & 1u) << 15));
  const __half d16 = __float2half_rn(__fmul_rn(ext, -0.125f));   // exact but for the fp16 rounding
  d_bits = __half_as_ushort(d16);
  const float d = __half2float(d16);
  uint32_t w = 0x88888888u;  // d == 0: every code stands for zero
  if (d != 0.0f) {
    float x[8], q[8];
    widen8(u, x);
    divide8(x, d, q);
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // clamp(rint(q) + 8, 0, 15): the sum's last bits are the code (1.5 * 2^23 rounds to integers)
      const float c = __fadd_rn(fminf(fmaxf(q[i], -8.0f), 7.0f), 12582920.0f);
      w |= (__float_as_uint(c) & 15u) << (4 * i);
    }
  }
  return w;
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

// What a block covers: kUnroll rounds of `wide` neighbouring tokens of one sequence, `per` threads (eight
// elements each) a token; a token of more threads than the block has takes `turns`.  blockIdx.y: 0 = K,
// 1 = V; blockIdx.z: the sequence.
struct Shape {
  int per, wide, turns;
};

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvMoveArgs a, const Shape s) {
  const int which = blockIdx.y, tok = threadIdx.x / s.per, i0 = blockIdx.x * s.wide * kUnroll;
  const float g = FMT == WQ_NVFP4 && a.kv.g[which] ? *a.kv.g[which] : 1.0f;
  for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const int n = kv::count_of(a.counts, b, a.tokens);
    if (i0 >= n) continue;
    const int64_t start = kv::first_of(a.start, b);
    for (int turn = 0; turn < s.turns; ++turn) {
      const int c = threadIdx.x - tok * s.per + turn * (int)blockDim.x;
      const bool mine = tok < s.wide && c < s.per;
      const int h = c / (D / 8), e = (c % (D / 8)) * 8;
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.x[which].p) + b * a.x[which].batch + h * a.x[which].head + e;
      uint4 u[kUnroll];
      int64_t row[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + k * s.wide + tok;
        u[k] = make_uint4(0, 0, 0, 0);
        row[k] = -1;
        if (mine && i < n) {
          u[k] = *reinterpret_cast<const uint4*>(src + i * a.x[which].token);
          row[k] = kv::row_of(a.kv, b, start + i, h);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (i0 + k * s.wide >= n) break;      // for the whole block: its lanes exchange values below
        const uint32_t v[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        uint32_t w;
        uint16_t d = 0;
        uint8_t sb = 0;
        if (FMT == WQ_Q4_0) w = encode_q4_0(v, threadIdx.x & 31, d);
        else w = encode_nvfp4(v, g, sb);
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
}

template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvMoveArgs a, const Shape s) {
  const int which = a.x[0].p ? blockIdx.y : 1, tok = threadIdx.x / s.per, i0 = blockIdx.x * s.wide * kUnroll;
  const float g = FMT == WQ_NVFP4 && a.kv.g[which] ? *a.kv.g[which] : 1.0f;
  if (tok >= s.wide) return;
  for (int64_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
    const int n = kv::count_of(a.counts, b, a.tokens);
    const int64_t start = kv::first_of(a.start, b);
    for (int c = threadIdx.x - tok * s.per; c < s.per; c += s.turns > 1 ? (int)blockDim.x : s.per) {
      const int h = c / (D / 8), e = (c % (D / 8)) * 8;
      uint32_t w[kUnroll];
      float sc[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + k * s.wide + tok;
        w[k] = FMT == WQ_Q4_0 ? 0x88888888u : 0u;    // a row that is not there reads as zero
        sc[k] = 0.0f;
        const int64_t row = i < n ? kv::row_of(a.kv, b, start + i, h) : -1;
        if (row >= 0) {
          w[k] = *reinterpret_cast<const uint32_t*>(a.kv.codes[which] + row * (D / 2) + e / 2);
          sc[k] = kv::scale_at<FMT>(a.kv.scales[which] + row * kv::scale_bytes(D), e);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + k * s.wide + tok;
        if (i >= a.tokens) break;
        float v[8];
        kv::decode8<FMT>(w[k], sc[k], g, v);
        const int64_t at = b * a.x[which].batch + i * a.x[which].token + h * a.x[which].head + e;
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
}

struct Grid {
  Shape s;
  dim3 blocks, threads;
};
Grid grid_for(const KvMoveArgs& a, int sides) {
  Grid g{};
  g.s.per = a.kv.heads * (a.kv.dim / 8);
  const int64_t wide = g.s.per >= kThreads ? 1 : kThreads / g.s.per;
  g.s.wide = (int)(wide < a.tokens ? wide : a.tokens);
  const int threads = g.s.wide * g.s.per;
  g.threads = dim3((unsigned)(threads > kThreads ? kThreads : (threads + 31) / 32 * 32));
  g.s.turns = (int)((g.s.per + g.threads.x - 1) / g.threads.x);
  const int64_t step = (int64_t)g.s.wide * kUnroll;
  g.blocks = dim3((unsigned)((a.tokens + step - 1) / step), (unsigned)sides, (unsigned)(a.batch < 65535 ? a.batch : 65535));
  return g;
}

int launched() {
  count_launch();
  return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

template <int FMT, int D>
int append_t(const KvMoveArgs& a, cudaStream_t s) {
  const Grid g = grid_for(a, 2);
  kv_append_kernel<FMT, D><<<g.blocks, g.threads, 0, s>>>(a, g.s);
  return launched();
}
template <int FMT, int D>
int read_t(const KvMoveArgs& a, cudaStream_t s) {
  const Grid g = grid_for(a, (a.x[0].p ? 1 : 0) + (a.x[1].p ? 1 : 0));
  if (a.f32) kv_read_kernel<FMT, D, true><<<g.blocks, g.threads, 0, s>>>(a, g.s);
  else kv_read_kernel<FMT, D, false><<<g.blocks, g.threads, 0, s>>>(a, g.s);
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
