// wq_attend.cu -- attention over the 4-bit KV cache.
//
// One block per query row and head; its warps take the visible tokens in turn, each lane D / 32
// elements of a token.  Online softmax: m the running maximum of the scores (in base 2), l the sum
// of 2^(s - m), o the sum of 2^(s - m) v; warps are joined at the end, in order.
#include <cuda_runtime.h>

#include "wq_kv.cuh"

namespace wq {
namespace {

constexpr int kWarps = 4;

template <int FMT, int D>
__global__ void __launch_bounds__(32 * kWarps) attend_kernel(AttendArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / (uint32_t)a.tokens;
  const int i = (int)(blockIdx.x - (uint32_t)b * (uint32_t)a.tokens);
  const int hq = blockIdx.y, h = hq / (int)(a.q_heads / a.kv.heads);
  const int n = kv::count_of(a.counts, b, a.tokens);
  int len = max(a.lens[b], 0);
  if (len > a.kv.capacity) {
    if (threadIdx.x == 0) set_status(WQ_STATUS_ARG);
    len = (int)a.kv.capacity;
  }
  int lo = 0, hi = len;
  const int64_t p = (int64_t)len - n + i;
  if (a.causal) hi = (int)min((int64_t)hi, p + 1);
  if (a.window) lo = (int)max((int64_t)0, p - a.window + 1);
  if (i >= n) hi = 0;
  float q[E], o[E];
  const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q.p) + b * a.q.batch + i * a.q.token + hq * a.q.head;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    q[j] = bf16_bits_to_f32(qp[lane * E + j]);
    o[j] = 0.0f;
  }
  const float kg = FMT == WQ_NVFP4 && a.kv.g[0] ? *a.kv.g[0] : 1.0f, vg = FMT == WQ_NVFP4 && a.kv.g[1] ? *a.kv.g[1] : 1.0f;
  const float c = a.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.0f;
  for (int t = lo + warp; t < hi; t += kWarps) {
    const int64_t row = kv::row_of(a.kv, b, t, h);
    if (row < 0) continue;
    float k[8], v[8];
    const int e = lane * E, sh = 4 * (e & 7);
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(a.kv.codes[0] + row * (D / 2) + (e & ~7) / 2);
    const uint32_t vw = *reinterpret_cast<const uint32_t*>(a.kv.codes[1] + row * (D / 2) + (e & ~7) / 2);
    kv::decode8<FMT>(kw >> sh, kv::scale_at<FMT>(a.kv.scales[0] + row * kv::scale_bytes(D), e), kg, k);
    kv::decode8<FMT>(vw >> sh, kv::scale_at<FMT>(a.kv.scales[1] + row * kv::scale_bytes(D), e), vg, v);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) s = fmaf(q[j], k[j], s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s *= c;
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = fmaf(l, f, w);
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] = fmaf(o[j], f, w * v[j]);
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
  for (int j = 0; j < E; ++j) so[warp][lane * E + j] = o[j];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float top = -INFINITY, sum = 0.0f, out = 0.0f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float f = sl[w] == 0.0f ? 0.0f : exp2f(sm[w] - top);
    sum = fmaf(sl[w], f, sum);
    out = fmaf(so[w][threadIdx.x], f, out);
  }
  out = sum == 0.0f ? 0.0f : out / sum;
  const int64_t at = b * a.out.batch + i * a.out.token + hq * a.out.head + threadIdx.x;
  if (a.f32) reinterpret_cast<float*>(a.out.p)[at] = out;
  else reinterpret_cast<__nv_bfloat16*>(a.out.p)[at] = __float2bfloat16_rn(out);
  if (a.lse && threadIdx.x == 0)
    a.lse[(b * a.tokens + i) * a.q_heads + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int FMT, int D>
int attend_t(const AttendArgs& a, cudaStream_t s) {
  attend_kernel<FMT, D><<<dim3((unsigned)(a.batch * a.tokens), (unsigned)a.q_heads), 32 * kWarps, 0, s>>>(a);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? WQ_OK : WQ_ERR_CUDA;
}

}  // namespace

size_t attend_workspace(const KvArgs&, int64_t, int64_t, int64_t, int64_t) { return 0; }

int attend(const AttendArgs& a, cudaStream_t s) {
  if (a.kv.fmt == WQ_Q4_0) return a.kv.dim == 64 ? attend_t<WQ_Q4_0, 64>(a, s) : attend_t<WQ_Q4_0, 128>(a, s);
  return a.kv.dim == 64 ? attend_t<WQ_NVFP4, 64>(a, s) : attend_t<WQ_NVFP4, 128>(a, s);
}

int take_status_attend() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
