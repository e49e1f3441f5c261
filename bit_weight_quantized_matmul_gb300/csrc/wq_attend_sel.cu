// wq_attend_sel.cu -- attention over the 4-bit KV cache, few query rows per cached head, for sinks and trees of drafted tokens: the
// kernel of wq_attend_few.cuh, whose tiles are those of the first tokens and then the window's, and whose masks are words of bits.
//
// Measured on GB300: 64 x 1 over 1000 .. 32000 behind a window of 4096 and 4 sinks, 32/8 heads of 128 (NVFP4), 77 us with the
// join (3.8 TB/s of 6.8 for a copy); 64 x 5 nodes over 1000 .. 16000 274 us; one token over 2000 behind
// 256 of 20 heads of 64 7 us, bound by its dependent loads.
#include "wq_attend_few.cuh"

namespace wq {

int attend_few_sel(const AttendArgs& a, const AttendFewPlan& pl, cudaStream_t s) { return launch_few<true>(a, pl, s); }

int take_status_attend_few_sel() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
