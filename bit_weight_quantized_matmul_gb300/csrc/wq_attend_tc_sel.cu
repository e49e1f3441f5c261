// wq_attend_tc_sel.cu -- the same for sinks and trees of drafted tokens.
#include "wq_attend_tc.cuh"

namespace wq {

int attend_tc_sel(const AttendArgs& a, const AttendTcPlan& pl, cudaStream_t s) { return launch_tc<true>(a, pl, s); }

int take_status_attend_tc_sel() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return WQ_ERR_CUDA;
  cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
  return v;
}

}  // namespace wq
