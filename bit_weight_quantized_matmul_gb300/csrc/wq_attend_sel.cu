// wq_attend_sel.cu -- attention over the 4-bit KV cache, few query rows per cached head, for sinks and trees of drafted tokens.
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
