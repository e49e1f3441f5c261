// wq_kv.cu -- quantising rows into the 4-bit KV cache as they are written, and reading them back.
//
// Both move each element once; HBM bounds them (append: 2 bytes in, 9/16 out; read the other way
// round), and the launch a call of few tokens.  A block owns one token and a thread eight
// elements of a head: one 16-byte access on the bf16 side, four bytes of codes.  A q4_0 block is
// then four neighbouring lanes, an NVFP4 block two, and the block's scale a maximum over them.
#include <cuda_runtime.h>

#include "wq_kv.cuh"

namespace wq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const uint16_t* p, uint32_t (&u)[4]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
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
  const __half d16 = __float2half_rn(__fdiv_rn(ext, -8.0f));
  d_bits = __half_as_ushort(d16);
  const float d = __half2float(d16);
  uint32_t w = 0x88888888u;  // d == 0: every code stands for zero
  if (d != 0.0f) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = bf16_bits_to_f32((u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
      const float q = fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(x, d)), 8.0f), 0.0f), 15.0f);
      w |= (uint32_t)q << (4 * i);
    }
  }
  return w;
}

// Codes of eight bf16 values of an NVFP4 block (two lanes hold its 16) and its E4M3 scale.
__device__ __forceinline__ uint32_t encode_nvfp4(const uint32_t (&u)[4], float g, uint8_t& s_byte) {
  float x[8], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = bf16_bits_to_f32((u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  const uint32_t s = f32_to_e4m3_cvt(__fdiv_rn(__fdiv_rn(amax, 6.0f), g));
  s_byte = (uint8_t)s;
  const float S = __fmul_rn(e4m3_to_f32(s), g);
  if (S == 0.0f) return 0u;  // a block whose scale underflows keeps codes 0
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], S);
  return f32x8_to_e2m1x8(x);
}

// One token: eight elements of every head of K, then of V, per thread and round.
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvMoveArgs a) {
  constexpr int kChunks = D / 8;
  const int64_t b = blockIdx.x / (uint32_t)a.tokens;
  const int i = (int)(blockIdx.x - (uint32_t)b * (uint32_t)a.tokens);
  if (i >= kv::count_of(a.counts, b, a.tokens)) return;
  const int t = kv::first_of(a.start, b) + i;
  const int64_t row0 = t < 0 ? -1 : kv::row_of(a.kv, b, t, 0);
  if (row0 < 0) {
    if (t < 0) set_status(WQ_STATUS_ARG);
    return;
  }
  const int per = a.kv.heads * kChunks, total = 2 * per;
  // rounds cover whole warps, so that the lanes of a quantisation block stay together
  for (int it = threadIdx.x; it < ((total + 31) & ~31); it += kThreads) {
    const bool in = it < total;
    const int which = in && it >= per;
    const int j = in ? it - which * per : 0;
    const int h = j / kChunks, e = (j % kChunks) * 8;
    uint32_t u[4] = {0, 0, 0, 0};
    if (in)
      load8(reinterpret_cast<const uint16_t*>(a.x[which].p) + b * a.x[which].batch + i * a.x[which].token +
                h * a.x[which].head + e, u);
    const int64_t row = row0 + (int64_t)h * a.kv.page_size;
    uint32_t w;
    if (FMT == WQ_Q4_0) {
      uint16_t d;
      w = encode_q4_0(u, threadIdx.x & 31, d);
      if (in && (e & 31) == 0) reinterpret_cast<uint16_t*>(a.kv.scales[which])[row * (D / 32) + e / 32] = d;
    } else {
      const float g = a.kv.g[which] ? *a.kv.g[which] : 1.0f;
      uint8_t s;
      w = encode_nvfp4(u, g, s);
      if (in && (e & 15) == 0) a.kv.scales[which][row * (D / 16) + e / 16] = s;
    }
    if (in) *reinterpret_cast<uint32_t*>(a.kv.codes[which] + row * (D / 2) + e / 2) = w;
  }
}

// One token: eight elements of every head of the wanted tensors per thread and round.
template <int FMT, int D, bool F32>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvMoveArgs a) {
  constexpr int kChunks = D / 8;
  const int64_t b = blockIdx.x / (uint32_t)a.tokens;
  const int i = (int)(blockIdx.x - (uint32_t)b * (uint32_t)a.tokens);
  int64_t row0 = -1;
  if (i < kv::count_of(a.counts, b, a.tokens)) {
    const int t = kv::first_of(a.start, b) + i;
    if (t >= 0) row0 = kv::row_of(a.kv, b, t, 0);
    else set_status(WQ_STATUS_ARG);
  }
  const int per = a.kv.heads * kChunks;
  const int begin = a.x[0].p ? 0 : per, end = a.x[1].p ? 2 * per : per;
  for (int it = begin + threadIdx.x; it < end; it += kThreads) {
    const int which = it >= per;
    const int j = it - which * per;
    const int h = j / kChunks, e = (j % kChunks) * 8;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row0 >= 0) {
      const int64_t row = row0 + (int64_t)h * a.kv.page_size;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(a.kv.codes[which] + row * (D / 2) + e / 2);
      const float s = kv::scale_at<FMT>(a.kv.scales[which] + row * kv::scale_bytes(D), e);
      kv::decode8<FMT>(w, s, FMT == WQ_NVFP4 && a.kv.g[which] ? *a.kv.g[which] : 1.0f, v);
    }
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

int launched() {
  count_launch();
  return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

template <int FMT, int D>
int append_t(const KvMoveArgs& a, cudaStream_t s) {
  kv_append_kernel<FMT, D><<<(unsigned)(a.batch * a.tokens), kThreads, 0, s>>>(a);
  return launched();
}
template <int FMT, int D>
int read_t(const KvMoveArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(a.batch * a.tokens);
  if (a.f32) kv_read_kernel<FMT, D, true><<<grid, kThreads, 0, s>>>(a);
  else kv_read_kernel<FMT, D, false><<<grid, kThreads, 0, s>>>(a);
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
