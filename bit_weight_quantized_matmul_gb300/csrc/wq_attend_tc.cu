// wq_attend_tc.cu -- attention over the 4-bit KV cache, many query rows per cached head (wq_attend_tc.cuh).
#include "wq_attend_tc.cuh"

namespace wq {

int attend_tc(const AttendArgs& a, const AttendTcPlan& pl, cudaStream_t s) { return launch_tc<false>(a, pl, s); }

int take_status_attend_tc() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
